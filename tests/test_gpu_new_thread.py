"""A host thread whose first CUDA work is a call of the library: nothing on it has
made the device's context current, and what the library keeps per device is there
already from calls on another thread."""
import ctypes
import threading

import pytest
import torch

import selective_state_space_mss_b200 as mss
from selective_state_space_mss_b200 import inputs as gen
from tests.helpers import device_inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _scan(batch, dim, L, dtype="bf16"):
    return device_inputs(gen.scan_inputs(batch, dim, 16, L, dtype, seed=700, d_skip="normal"), DEV)


def _rnd(*s, dt=torch.bfloat16):
    return torch.randn(*s, generator=torch.Generator().manual_seed(len(s))).to(DEV, dt)


def _scan_step():
    d = _scan(2, 64, 512)
    dy = _rnd(2, 64, 512)

    def run():
        y, last, states = mss.scan_fwd_save(**d)
        g = mss.scan_bwd(dy=dy, saved_states=states, **d)
        # the others are summed with atomics: their bits may differ between any two calls
        return dict(y=y, last=last, **{k: g[k] for k in ("du", "ddelta", "dz")})
    return run


def _glr_step(dt, off):
    B, L, D = (1, 200, 64) if off else (2, 200, 64)
    x, gate, z, dy = (_rnd(B, L, D, dt=dt) for _ in range(4))
    kw = dict(z=z, seq_offsets=torch.tensor(off, dtype=torch.int32, device=DEV) if off else None)

    def run():
        y, last, states = mss.glr_fwd_save(x, gate, **kw)
        return dict(mss.glr_bwd(x, gate, dy, saved_states=states, **kw), y=y, last=last)
    return run


def _glr_token():
    state, x, gate = _rnd(3, 64, dt=torch.float32), _rnd(3, 64), _rnd(3, 64)

    def run():
        out = torch.empty_like(state)
        return dict(y=mss.glr_update(state, x, gate, state_out=out), state=out)
    return run


def _norm(dim):
    x, w, dy = _rnd(300, dim), torch.ones(dim, device=DEV), _rnd(300, dim)

    def run():
        y, _, mean, rstd = mss.norm_fwd(x, w)
        return dict(mss.norm_bwd(x, w, dy, rstd, mean=mean), y=y, mean=mean, rstd=rstd)
    return run


def _ssd(n):
    x, dt = _rnd(1, 300, 4, 64), _rnd(1, 300, 4)
    A, B, C = -torch.rand(4, device=DEV) - 0.5, _rnd(1, 300, 1, n), _rnd(1, 300, 1, n)
    return lambda: dict(zip("ys", mss.ssd_fwd(x, dt, A, B, C)))


CALLS = {
    "scan": lambda: (lambda d: lambda: dict(zip("ys", mss.scan_fwd(**d, flags=mss.FLAG_PAIR_LANES))))(_scan(2, 64, 512)),
    "scan, four lanes": lambda: (lambda d: lambda: dict(zip("ys", mss.scan_fwd(**d))))(_scan(2, 64, 512)),
    "scan, training step": _scan_step,
    "ssd, 64": lambda: _ssd(64),
    "ssd, 128": lambda: _ssd(128),
    "recurrence, bf16": lambda: _glr_step(torch.bfloat16, None),
    "recurrence, fp32 packed": lambda: _glr_step(torch.float32, [0, 50, 51, 200]),
    "recurrence, token": _glr_token,
    "norm, whole words": lambda: _norm(96),
    "norm, parts of words": lambda: _norm(101),
}


@pytest.mark.parametrize("name", CALLS)
def test_first_cuda_work_of_a_thread(name):
    run = CALLS[name]()
    for _ in range(3):  # the allocator keeps what the thread's call takes: no allocation makes a context current
        want = run()
    want = {k: v.clone() for k, v in want.items() if v is not None}
    again = run()
    del again
    torch.cuda.synchronize()
    got, failed = [], []

    def work():
        try:
            ctx = ctypes.c_void_p()
            assert ctypes.CDLL("libcuda.so.1").cuCtxGetCurrent(ctypes.byref(ctx)) == 0 and not ctx.value
            got.append(run())
            torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001 -- reported by the test
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    assert mss.get_device_error() == 0
    for k, v in want.items():
        assert torch.equal(got[0][k], v), k
