"""Rows of no elements: their statistics are the quotients 0 / 0."""
import pytest
import torch

import selective_state_space_mss_b200 as mss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("residual", [False, True], ids=["x", "x+residual"])
def test_statistics_of_rows_without_elements(residual, rms):
    held = torch.full((2, 3), 7.0, device=DEV)  # what the allocator hands on next is not 0 / 0
    del held
    x, w = torch.zeros(2, 3, 0, dtype=torch.bfloat16, device=DEV), torch.zeros(0, device=DEV)
    y, s, mean, rstd = mss.norm_fwd(x, w, residual=x.float() if residual else None, rms=rms)
    assert y.shape == x.shape and (s.shape == x.shape if residual else s is None)
    assert rstd.shape == (2, 3) and torch.isnan(rstd).all()
    assert mean is None if rms else mean.shape == (2, 3) and torch.isnan(mean).all()
    assert mss.norm_fwd(x, w, rms=rms, want_stats=False)[2:] == (None, None)
    stream = torch.cuda.Stream(DEV)
    _, _, _, rstd = mss.norm_fwd(x, w, rms=rms, stream=stream)
    stream.synchronize()
    assert torch.isnan(rstd).all()
    g = mss.norm_bwd(x, w, x, rstd, mean=None if rms else rstd)
    assert g["dx"].shape == x.shape and g["dweight"].shape == (0,)
