"""The give-up paths of the recurrence's and the norm's kernels, without a fault: in
the library's self-test each kernel waits for its first tiles or rows with a limit
of 1 ms, and their barriers complete only when the waits have given up.  The error reaches the
host once, nothing outside the outputs is written, and the next calls are right to
the bit."""
import threading

import pytest
import torch

import selective_state_space_mss_b200 as mss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def selftest():
    assert mss.get_device_error() == 0

    def run(call):
        assert mss.selftest_timeout(True) is False
        try:
            return call()
        finally:
            assert mss.selftest_timeout(False) is True

    return run


def _guarded(like):
    """An output like `like` between two margins of sevens."""
    raw = torch.full((like.numel() + 128,), 7.0, dtype=like.dtype, device=DEV)
    return raw, raw[64:64 + like.numel()].view(like.shape)


def _margins(raw):
    assert (raw[:64] == 7).all() and (raw[-64:] == 7).all()


def _same(a, b):
    for k, v in a.items():
        assert v is None and b[k] is None or torch.equal(v, b[k]), k


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
# one block a sequence, clusters, more units than blocks at once, packed
@pytest.mark.parametrize("size", [(1, 64, 64, None), (2, 300, 72, None), (400, 70, 64, None), (1, 500, 128, [0, 30, 31, 200, 500])], ids=str)
@pytest.mark.parametrize("z", [True, False], ids=["z", "plain"])
def test_recurrence(selftest, size, z, dt):
    B, L, D, off = size
    gen = torch.Generator(device=DEV).manual_seed(L)
    x, gate, zz, dy = (torch.randn(B, L, D, generator=gen, device=DEV).to(dt) for _ in range(4))
    kw = dict(z=zz if z else None, seq_offsets=None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV))

    def forward(y=None):
        y, last, states = mss.glr_fwd_save(x, gate, y=y, **kw)
        return dict(y=y, last=last, states=states)

    want = forward()
    grads = mss.glr_bwd(x, gate, dy, saved_states=want["states"], **kw)
    raw, y = _guarded(x)
    selftest(lambda: forward(y))
    assert mss.get_device_error() == mss.ERR_DEVICE_TIMEOUT and mss.get_device_error() == 0
    assert (raw == 7).all()  # given up before the first output
    _same(want, forward())
    outs = {k: _guarded(x) for k in ("dx", "dgate") + (("dz",) if z else ())}
    selftest(lambda: mss.glr_bwd(x, gate, dy, saved_states=want["states"], out={k: v[1] for k, v in outs.items()}, **kw))
    assert mss.get_device_error() == mss.ERR_DEVICE_TIMEOUT and mss.get_device_error() == 0
    for raw, _ in outs.values():
        assert (raw == 7).all()
    _same(grads, mss.glr_bwd(x, gate, dy, saved_states=want["states"], **kw))
    assert mss.get_device_error() == 0


@pytest.mark.parametrize("types", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)],
                         ids=["f32", "bf16+f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
# rows of whole and of parts of words, fewer and more of them than groups, one and more warps a row
@pytest.mark.parametrize("size", [(3, 64), (2000, 96), (700, 768), (3, 101), (2000, 101), (700, 1001), (160, 8191)], ids=str)
def test_norm(selftest, size, rms, types):
    dt, st = types
    gen = torch.Generator(device=DEV).manual_seed(sum(size))
    rnd = lambda t: torch.randn(*size, generator=gen, device=DEV).to(t)
    x, res, dy, dres, w = rnd(dt), rnd(st), rnd(dt), rnd(st), torch.randn(size[1], generator=gen, device=DEV)
    forward = lambda **kw: dict(zip(("y", "s", "mean", "rstd"), mss.norm_fwd(x, w, residual=res, rms=rms, **kw)))
    want = forward()
    back = lambda **kw: mss.norm_bwd(want["s"], w, dy, want["rstd"], mean=want["mean"], dresidual=dres, **kw)
    grads = back()
    if size[1] % 8 == 0:  # the forward pass has no waits
        with pytest.raises(mss.MssError) as e:
            selftest(forward)
        assert e.value.code == mss.ERR_FLAGS
    else:
        (ry, y), (rs, s) = _guarded(x), _guarded(res)
        selftest(lambda: forward(y=y, residual_out=s))
        assert mss.get_device_error() == mss.ERR_DEVICE_TIMEOUT
        assert (ry == 7).all()
        _margins(rs)
    assert mss.get_device_error() == 0
    _same(want, forward())
    raw, dx = _guarded(x)
    selftest(lambda: back(out=dict(dx=dx)))
    assert mss.get_device_error() == mss.ERR_DEVICE_TIMEOUT and mss.get_device_error() == 0
    assert (raw == 7).all()
    _same(grads, back())
    assert mss.get_device_error() == 0


def test_calls_without_waits_are_refused_and_other_threads_are_not_touched(selftest):
    x = torch.randn(2, 100, 33, device=DEV)  # rows that are not whole 16-byte pieces
    w = torch.ones(8200, device=DEV)
    wide, r = torch.randn(4, 8200, device=DEV), torch.ones(4, device=DEV)
    for call in (lambda: mss.glr_fwd(x, x), lambda: mss.norm_bwd(wide, w, wide, r), lambda: mss.norm_fwd(wide, w)):
        with pytest.raises(mss.MssError) as e:
            selftest(call)
        assert e.value.code == mss.ERR_FLAGS
        call()
    y = torch.randn(2, 100, 64, device=DEV)
    got = []

    def both():
        t = threading.Thread(target=lambda: got.append(mss.glr_fwd(y, y)[0]))
        t.start()
        t.join()

    selftest(both)
    assert mss.get_device_error() == 0 and torch.equal(got[0], mss.glr_fwd(y, y)[0])
