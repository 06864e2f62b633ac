"""Which gradients the recurrence's and the norm's backward passes return: every
one that was asked for, in its shape and type, and written."""
import pytest
import torch

import selective_state_space_mss_b200 as mss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _written(v, shape, dtype, what):
    assert v is not None and v.shape == shape and v.dtype == dtype and v.device == torch.device(DEV), what
    assert torch.isfinite(v).all() and (v != 0).any(), what


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("z", [False, True], ids=["plain", "z"])
@pytest.mark.parametrize("optional", [False, True], ids=["none", "bias+init+dlast"])
@pytest.mark.parametrize("saved", [False, True], ids=["recomputed", "saved"])
@pytest.mark.parametrize("want", [(True, True), (True, False), (False, True), (False, False)], ids=str)
def test_recurrence(want, saved, optional, z, packed, dt):
    gen = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s, t=dt: torch.randn(*s, generator=gen, device=DEV).to(t)
    B, L, D = (1, 150, 72) if packed else (3, 150, 72)
    n = 4 if packed else B
    kw = dict(z=rnd(B, L, D) if z else None, gate_bias=rnd(D, t=torch.float32) if optional else None,
              initial_state=rnd(n, D, t=torch.float32) if optional else None,
              seq_offsets=torch.tensor([0, 20, 90, 91, L], dtype=torch.int32, device=DEV) if packed else None)
    x, gate, dy = (rnd(B, L, D) for _ in range(3))
    y, last, states = mss.glr_fwd_save(x, gate, **kw)
    _written(y, x.shape, dt, "y")
    _written(last, (n, D), torch.float32, "last")
    got = mss.glr_bwd(x, gate, dy, **kw, dlast=rnd(n, D, t=torch.float32) if optional else None,
                      saved_states=states if saved else None, want_dbias=want[0], want_dinit=want[1])
    shapes = dict(dx=(x.shape, dt), dgate=(x.shape, dt), dz=(x.shape, dt) if z else None,
                  dbias=((D,), torch.float32) if want[0] else None, dinit=((n, D), torch.float32) if want[1] else None)
    assert set(got) == set(shapes)
    for k, v in shapes.items():
        if v is None:
            assert got[k] is None, k
        else:
            _written(got[k], *v, k)


@pytest.mark.parametrize("types", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)],
                         ids=["f32", "bf16+f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("want", [(True, True), (True, False), (False, True), (False, False)], ids=str)
def test_norm(want, rms, types):
    dt, st = types
    gen = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s, t=torch.float32: torch.randn(*s, generator=gen, device=DEV).to(t)
    w = 1 + 0.1 * rnd(72)
    y, s, mean, rstd = mss.norm_fwd(rnd(50, 72, t=dt), w, residual=rnd(50, 72, t=st), rms=rms)
    _written(y, (50, 72), dt, "y")
    _written(s, (50, 72), st, "s")
    got = mss.norm_bwd(s, w, rnd(50, 72, t=dt), rstd, mean=mean, dresidual=rnd(50, 72, t=st), want_dweight=want[0], want_dbias=want[1])
    shapes = dict(dx=((50, 72), dt), dresidual=((50, 72), st) if st != dt else None,
                  dweight=((72,), torch.float32) if want[0] else None, dbias=((72,), torch.float32) if want[1] else None)
    assert set(got) == set(shapes)
    for k, v in shapes.items():
        if v is None:
            assert got[k] is None, k
        else:
            _written(got[k], *v, k)
