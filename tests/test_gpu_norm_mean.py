"""The norm's backward pass where the mean is far above the spread: x^ = (s -
mean) rstd with the difference taken first, whose rounding is relative to the
difference, not to the mean.

U = 2^-24 is the half step of fp32: the difference, the product with rstd and
the few operations on it round by U of their own size each.
"""
import pytest
import torch

import selective_state_space_mss_b200 as mss

from tests import recurrent_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def gradients(s, weight, dy, mean, rstd, dres, out, s_out):
    """float64, mean and rstd as the kernel is given them; {name: (value, bound)}."""
    n, r = s.shape[1], rstd[:, None]
    hat = (s - mean[:, None]) * r
    ehat = hat.abs() * 3 * U
    g = dy * weight
    adds = (n / 256 + 40) * U  # additions in a row, of a thread and of the tree over the row's threads
    a, b = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    ea = g.abs().mean(1, keepdim=True) * (adds + 2 * U)
    eb = (g.abs() * ehat).mean(1, keepdim=True) + (g * hat).abs().mean(1, keepdim=True) * (adds + 3 * U)
    d = r * (g - a - hat * b)
    ed = r * (ea + ehat * b.abs() + hat.abs() * eb + (g.abs() + a.abs() + (hat * b).abs()) * 8 * U)
    if dres is not None:
        d, ed = d + dres, ed + (d.abs() + dres.abs()) * 2 * U
    rows = (s.shape[0] - 1) * U  # additions of values other than 0
    return dict(dx=(d, ed + d.abs() * ref.half_step(out)), dresidual=(d, ed + d.abs() * ref.half_step(s_out)),
                dweight=((dy * hat).sum(0), (dy.abs() * ehat).sum(0) + (dy * hat).abs().sum(0) * (rows + 3 * U)),
                dbias=(dy.sum(0), dy.abs().sum(0) * rows))


@pytest.mark.parametrize("types", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)],
                         ids=["f32", "bf16+f32", "bf16"])
# rows of whole words, of parts of words, from between words, and past the registers
@pytest.mark.parametrize("form", [(1024, 0), (64, 0), (1001, 0), (5, 0), (300, 1), (1024, 1), (8200, 0)], ids=str)
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("mean", [10.0, -1000.0, 1e5])
def test_mean_above_the_spread(mean, rows, form, types):
    dim, front = form
    dt, st = types
    gen = torch.Generator().manual_seed(dim + rows)
    rnd = lambda *sh: torch.randn(*sh, generator=gen)
    s = (rnd(rows, dim) + mean).to(st)
    w, dy, dres = 1 + 0.3 * rnd(dim), rnd(rows, dim).to(dt), rnd(rows, dim).to(st)
    m = s.double().mean(1).float()
    r = (((s.double() - m.double()[:, None]) ** 2).mean(1) + 1e-5).rsqrt().float()

    def put(v):
        raw = torch.empty(v.numel() + front, dtype=v.dtype, device=DEV)
        raw[front:] = v.reshape(-1).to(DEV)
        return raw[front:].view(v.shape)

    got = mss.norm_bwd(put(s), w.to(DEV), put(dy), r.to(DEV), mean=m.to(DEV), dresidual=put(dres))
    want = gradients(s.double(), w.double(), dy.double(), m.double(), r.double(), dres.double(), dt, st)
    for k, v in got.items():
        if v is None:
            assert k == "dresidual" and dt == st
        else:
            ref.check(v, want[k], k)
