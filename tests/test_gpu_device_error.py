"""mss_get_device_error where a wait gave up and packed offsets broke their rule
before it was asked: each is reported, once."""
import pytest
import torch

import selective_state_space_mss_b200 as mss
from selective_state_space_mss_b200 import inputs as gen
from tests.helpers import device_inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("timeout_first", [True, False])
def test_both_errors_are_reported(timeout_first):
    assert mss.get_device_error() == 0
    d = device_inputs(gen.scan_inputs(2, 64, 16, 512, "bf16", seed=700, d_skip="normal"), DEV)
    x = torch.randn(1, 100, 40, device=DEV)

    def timeout():
        mss.scan_fwd(**d, flags=mss.FLAG_SELFTEST_TIMEOUT)

    def offsets():
        mss.glr_fwd(x, x, seq_offsets=torch.tensor([0, 60, 30, 100], dtype=torch.int32, device=DEV))

    for call in (timeout, offsets) if timeout_first else (offsets, timeout):
        call()
    assert {mss.get_device_error(), mss.get_device_error()} == {mss.ERR_DEVICE_TIMEOUT, mss.ERR_OFFSETS}
    assert mss.get_device_error() == 0
    offsets()
    assert mss.get_device_error() == mss.ERR_OFFSETS and mss.get_device_error() == 0
    timeout()
    assert mss.get_device_error() == mss.ERR_DEVICE_TIMEOUT and mss.get_device_error() == 0
