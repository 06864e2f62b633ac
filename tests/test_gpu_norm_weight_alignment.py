"""The norm where only the parameters begin between 16-byte words: rows of whole
words whose weight and bias have to be read element by element."""
import pytest
import torch

import selective_state_space_mss_b200 as mss

from tests import recurrent_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("types", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)],
                         ids=["f32", "bf16+f32", "bf16"])
@pytest.mark.parametrize("size", [(3, 8), (1100, 64), (300, 768), (160, 2304), (150, 8192), (2, 8200)], ids=str)
def test_parameters_between_words(size, types):
    dt, st = types
    gen = torch.Generator().manual_seed(sum(size))
    rnd = lambda *s: torch.randn(*s, generator=gen)
    x, res, dy, dres = rnd(*size).to(dt), rnd(*size).to(st), rnd(*size).to(dt), rnd(*size).to(st)
    w, b = 1 + 0.3 * rnd(size[1]), rnd(size[1])
    between = lambda v: torch.cat([v.new_zeros(1), v]).to(DEV)[1:]
    out = dict(dweight=torch.full((size[1] + 1,), 7.0, device=DEV)[1:], dbias=torch.full((size[1] + 1,), 7.0, device=DEV)[1:])
    y, s, mean, rstd = mss.norm_fwd(x.to(DEV), between(w), bias=between(b), residual=res.to(DEV))
    want = ref.norm(x.double(), w.double(), b.double(), res.double(), out=dt, res_dtype=st)
    for k, v in dict(y=y, s=s, mean=mean, rstd=rstd).items():
        ref.check(v, want[k], k)
    got = mss.norm_bwd(s, between(w), dy.to(DEV), rstd, mean=mean, dresidual=dres.to(DEV), out=out)
    wg = ref.norm_grad(s.cpu().double(), w.double(), dy.double(), mean.cpu().double(), rstd.cpu().double(), dres.double(), out=dt, s_out=st)
    for k, v in got.items():
        if v is None:
            assert k == "dresidual" and dt == st
        else:
            ref.check(v, wg[k], k)
