"""The gated linear recurrence with gates over their whole range, forward,
backward and decode, against the definition in 64 bits.

U = 2^-24 is the half step of fp32.  A gate is formed from e = e^-v: the argument
v (times log2 e) is rounded up to three times, which is 3 |v| U in e's relative
size, and the exponential, the reciprocal and the products around them add at
most 16 U.  With s = sigmoid(v), an error r relative to e is s (1 - s) r in s and in
1 - s.  e may come out as 0 below 2^-126 and goes up to 2^124 at most, so either
gate is off by up to 2^-124 where it is smaller than that (LOW, with the roundings
of that border: 86 x 2 U and less in e); silu(z) stops where its gate does,
at z = -124 ln 2, so 87 LOW covers it from there on.
"""
import pytest
import torch

import selective_state_space_mss_b200 as mss

from tests import recurrent_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, TINY, LOW = 2.0 ** -24, 2.0 ** -126, 2.0 ** -123
TYPES = [torch.bfloat16, torch.float32]
IDS = ["bf16", "f32"]

# the lowest finite value stands for None; each value has a channel of its own
BELOW = [None, -1e20, -1e15, -1e10, -1e4, -200.0, -104.0, -95.0, -89.0, -87.0, -60.0, -45.0, -42.0, -41.0, -30.0, -17.0]
ABOVE = [17.0, 30.0, 41.0, 42.0, 60.0, 87.0, 104.0, 200.0, 1e4]


def sigmoid(v):
    """(s, error), (1 - s, error)."""
    s, n = torch.sigmoid(v), torch.sigmoid(-v)
    err = s * n * (3 * v.abs() + 16) * U + LOW
    return (s, err + s * 2 * U), (n, err + n * 2 * U)


def recurrence(x, gate, z, init, out, dy=None, dlast=None):
    """[batch, L, dim] float64; {name: (value, bound)}."""
    hs = ref.half_step(out)
    (f, ef), (w, ew) = sigmoid(gate)
    h, eh, before, ebefore = (torch.empty_like(x) for _ in range(4))
    c, e, m = init, torch.zeros_like(init), init.abs()  # m: the sum of the terms' sizes
    for t in range(x.shape[1]):
        before[:, t], ebefore[:, t] = c, e
        term = w[:, t] * x[:, t]
        e = f[:, t] * e + ef[:, t] * m + ew[:, t] * x[:, t].abs()
        c = f[:, t] * c + term
        m = f[:, t] * m + term.abs()
        e = e + m * 4 * U + (m + 1) * TINY
        h[:, t], eh[:, t] = c, e
    if z is None:
        si, esi = torch.ones_like(x), torch.zeros_like(x)
    else:
        (g, eg), (n, en) = sigmoid(z)
        si = z * g
        esi = torch.where(z < -85, torch.full_like(z, 87 * LOW), z.abs() * eg) + si.abs() * 2 * U
    y = h * si
    res = dict(y=(y, si.abs() * eh + h.abs() * esi + y.abs() * (hs + 4 * U) + TINY), last=(c, e))
    if dy is None:
        return res
    up, eup = dy * si, dy.abs() * esi + (dy * si).abs() * 2 * U
    dh, edh = torch.empty_like(x), torch.empty_like(x)
    c, e, m = dlast, torch.zeros_like(dlast), dlast.abs()
    for t in reversed(range(x.shape[1])):
        c, m = up[:, t] + c, up[:, t].abs() + m
        e = e + eup[:, t] + m * 4 * U
        dh[:, t], edh[:, t] = c, e
        e = f[:, t] * e + ef[:, t] * m + f[:, t] * m * 4 * U + (m + 1) * TINY
        c, m = f[:, t] * c, f[:, t] * m
    res["dinit"] = (c, e)
    dx = w * dh
    res["dx"] = (dx, w * edh + ew * dh.abs() + dx.abs() * (hs + 4 * U) + TINY)
    d, fw = before - x, f * w
    ed, efw = ebefore + (before.abs() + x.abs()) * 2 * U, f * ew + w * ef
    dg = dh * d * fw
    edg = edh * (d * fw).abs() + ed * (dh * fw).abs() + efw * (dh * d).abs() + dg.abs() * 8 * U + (1 + dh.abs()) * (1 + d.abs()) * TINY
    res["dgate"] = (dg, edg + dg.abs() * hs)
    rows = x.shape[0] * x.shape[1]
    res["dbias"] = (dg.sum((0, 1)), edg.sum((0, 1)) + dg.abs().sum((0, 1)) * rows * U)
    if z is not None:
        ds = g + si * n
        eds = eg + esi * n + si.abs() * en + (g.abs() + (si * n).abs()) * 4 * U
        dz = dy * h * ds
        res["dz"] = (dz, (dy * ds).abs() * eh + (dy * h).abs() * eds + dz.abs() * (hs + 8 * U) + TINY)
    return res


def _channels(values, dt, L, every, shift, gen, base):
    """[2, L, len(values)]: random tokens, and in every `every`-th one the channel's value."""
    v = torch.randn(2, L, len(values), generator=gen) + base
    row = torch.tensor([torch.finfo(dt).min if a is None else a for a in values])
    v[:, shift::every] = row
    return v.to(dt)


def _inputs(dt, L, gates, zs, size, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    D = len(gates or zs)
    d = dict(x=rnd(2, L, D).to(dt), gate=_channels(gates, dt, L, 9, 4, gen, 1.0) if gates else (rnd(2, L, D) + 1).to(dt),
             z=None if zs is None else _channels(zs, dt, L, 3, 1, gen, 0.0) if zs else rnd(2, L, D).to(dt),
             initial_state=rnd(2, D) * size)
    return d, dict(dy=rnd(2, L, D).to(dt), dlast=rnd(2, D))


def _pad(d, front):
    """The same tensors, `front` elements behind a 16-byte boundary."""
    def put(v):
        if v is None or v.dim() != 3:
            return None if v is None else v.to(DEV)
        raw = torch.empty(v.numel() + front, dtype=v.dtype, device=DEV)
        raw[front:] = v.reshape(-1).to(DEV)
        return raw[front:].view(v.shape)
    return {k: put(v) for k, v in d.items()}


def _check(d, g, dt, front=0):
    dbl = lambda v: None if v is None else v.double()
    gd, gg = _pad(d, front), _pad(g, front)
    y, last, states = mss.glr_fwd_save(**gd)
    got = dict(mss.glr_bwd(**gd, **gg, saved_states=states), y=y, last=last)
    want = recurrence(*(dbl(d[k]) for k in ("x", "gate", "z", "initial_state")), dt, dbl(g["dy"]), dbl(g["dlast"]))
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k, r in want.items():
        ref.check(got[k], r, k)
    # one token of the same channels: the first that holds the values
    t = 4 if (d["gate"][:, 4].abs() > 16).any() else 1
    one = {k: None if d[k] is None else d[k][:, t] for k in ("x", "gate", "z")}
    state = d["initial_state"].to(DEV)
    y1 = mss.glr_update(state, **{k: None if v is None else v.contiguous().to(DEV) for k, v in one.items()})
    w1 = recurrence(*(None if v is None else v[:, None].double() for v in one.values()), dbl(d["initial_state"]), dt)
    ref.check(y1[:, None], w1["y"], "token y")
    ref.check(state, w1["last"], "token state")


# rows by TMA (8 channels are whole 16-byte pieces), by pieces, element by element
FORMS = [(16, 0), (15, 0), (16, 1)]


@pytest.mark.parametrize("dt", TYPES, ids=IDS)
@pytest.mark.parametrize("form", FORMS, ids=["tma", "pieces", "elements"])
@pytest.mark.parametrize("values", [BELOW, ABOVE + BELOW[9:16]], ids=["low", "high"])
def test_output_gate(values, form, dt):
    """silu goes to 0 below, to z above, and so do the gradients through it."""
    d, g = _inputs(dt, 150, None, values[:form[0]], 1.0, 3)
    _check(d, g, dt, form[1])


@pytest.mark.parametrize("dt", TYPES, ids=IDS)
@pytest.mark.parametrize("form", FORMS, ids=["tma", "pieces", "elements"])
@pytest.mark.parametrize("z", ["none", "plain", "extreme"])
@pytest.mark.parametrize("size", [1.0, 1e12, 1e25])
@pytest.mark.parametrize("values", [BELOW, ABOVE + BELOW[9:16]], ids=["low", "high"])
def test_forget_gate(values, size, z, form, dt):
    """A state of any size is replaced where the gate says so, and held where it says that."""
    n = form[0]
    zs = dict(none=None, plain=[], extreme=(BELOW[::-1])[:n])[z]
    d, g = _inputs(dt, 150, values[:n], zs, size, 5)
    _check(d, g, dt, form[1])
