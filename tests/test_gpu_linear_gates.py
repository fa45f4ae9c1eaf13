"""GPU tests of the gradient of linear attention's decays, dg: every set of outputs, on a workspace
that holds nothing of an earlier call, and its digits in heads and at tokens that forget fast.

Tolerance of dg_t: dg_t is the sum of the pairs i < t <= j, and m_t the sum of the magnitudes of all
products in them.  Each product passes through the rounding of three-part operands, fp32 sums
one after another (rows, states over chunks, chunks), three factors and two decays: 32 roundings of
2^-24 together.  A decay is 2^e with e rounded to fp32, which puts it off by |e| ln 2 of them, the token's
own |g| and what else lies between i and j; two decays: 2 |g_t| 2^-24.  So (32 + 2 |g_t|) 2^-24 m_t.
One decay a head: the tokens of a chunk may be off alike, chunks are off independently of each other,
so the root of the sum of the squares of the chunks' tolerances."""
import itertools
import math

import pytest
import torch

from test_gpu_linear_attention import (BF, F16, F32, UNIT, backward, bounds_of, forward, inputs,  # noqa: F401
                                       inside_of, s4)

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dstate")


def poisoned(s4, x, S, offsets, fwd, drop=()):  # noqa: F811
    """``backward`` on a workspace whose every float is NaN before the call."""
    fwd[0].workspace().fill_(0xFF)
    return backward(s4, x, S, offsets, fwd=fwd, drop=drop)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("gates", ["token", "head"])
@pytest.mark.parametrize("T,offsets", [(20, None), (300, None), (320, [0, 0, 1, 320]), (500, [2, 460, 480, 500])])
@pytest.mark.parametrize("Hk,Hv", [(2, 2), (1, 2)])
def test_every_set_of_outputs(s4, dtype, gates, T, offsets, Hk, Hv):  # noqa: F811
    """Outputs that are left out change no bit of the others, whatever the workspace held."""
    S = 2 if offsets is None else 3
    tokens = S * T if offsets is None else T
    x = inputs(T, tokens, S, Hk, Hv, 24, 40, dtype, gates=gates)
    fwd = forward(s4, x, S, offsets, training=True)
    every = poisoned(s4, x, S, offsets, fwd)
    assert all(bool(torch.isfinite(t).all()) for t in every.values())
    for n in range(1, 5):
        for drop in itertools.combinations(NAMES, n):
            got = poisoned(s4, x, S, offsets, fwd, drop)
            assert all(torch.equal(got[m], every[m]) for m in NAMES if m not in drop), drop


def gates_reference(x, S, offsets=None, scale=0.7):
    """dg by tokens and m, the same sums over the magnitudes, in 64 bits: [tokens, Hv] both."""
    z = {n: None if t is None else t.double() for n, t in x.items()}
    tokens, Hk, dk = z["q"].shape
    Hv, dv = z["v"].shape[1:]
    heads = torch.arange(Hv) // (Hv // Hk)
    q, k, v, do = z["q"][:, heads], z["k"][:, heads], z["v"], z["dout"]
    a = z["g"].exp().expand(tokens, Hv)
    out = []
    for f in (lambda t: t, torch.abs):
        got = torch.zeros(tokens, Hv, dtype=torch.float64)
        rows = [f(t) for t in (q, k, v, do)]
        for s, (lo, hi) in enumerate(bounds_of(S, tokens, offsets)):
            before = [torch.zeros(Hv, dk, dv, dtype=torch.float64) if z["state"] is None else f(z["state"][s])]
            for t in range(lo, hi):
                before.append(before[-1] * a[t][:, None, None] + rows[1][t][:, :, None] * rows[2][t][:, None, :])
            Z = f(z["dstate_out"][s])
            for t in range(hi - 1, lo - 1, -1):
                Z = Z + scale * rows[0][t][:, :, None] * rows[3][t][:, None, :]
                got[t] = a[t] * (Z * before[t - lo]).sum((1, 2))
                Z = Z * a[t][:, None, None]
        out.append(got)
    return out


def uniform(seed, *shape):
    return torch.rand(*shape, generator=torch.Generator().manual_seed(seed))


def check_gates(s4, x, S, offsets=None):  # noqa: F811
    tokens, g = x["q"].shape[0], x["g"]
    fwd = forward(s4, x, S, offsets, training=True)
    got = poisoned(s4, x, S, offsets, fwd)["dg"].double().cpu()
    ref, m = gates_reference(x, S, offsets)
    lim = (32 + 2 * g.double().abs().clamp(max=150)) * UNIT * m + 2.0 ** -126
    if g.dim() == 1:
        ref = ref.sum(0)
        chunks = [c.sum(0) ** 2 for lo, hi in bounds_of(S, tokens, offsets) if hi > lo for c in lim[lo:hi].split(64)]
        lim = (sum(chunks) if chunks else torch.zeros_like(ref)) ** 0.5 + 2.0 ** -126
    else:
        at = inside_of(S, tokens, offsets)
        got, ref, lim = got[at], ref[at], lim[at]
    worst = (got - ref).abs() / lim
    assert bool((worst <= 1).all()), f"parts of the tolerance, by heads: {worst.reshape(-1, g.shape[-1]).amax(0).tolist()}"


HEADS = [0.0, -0.02, -0.1, -0.5, -1.0, -2.0, -4.0, -5.0, -8.0, -10.0, -12.0, -15.0, -16.0, -30.0]


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("gates", ["token", "head"])
@pytest.mark.parametrize("T,dk,dv", [(70, 32, 24), (600, 16, 32), (200, 5, 3), (150, 128, 64), (200, 24, 160)])
def test_heads_that_forget(s4, dtype, gates, T, dk, dv):  # noqa: F811
    """From heads that forget nothing to those that keep 1e-13 of a token: dg keeps its digits in each."""
    Hv = len(HEADS)
    x = inputs(T, T, 1, Hv, Hv, dk, dv, dtype)
    x["g"] = torch.tensor(HEADS) if gates == "head" else torch.tensor(HEADS) * (0.9 + 0.2 * uniform(T, T, Hv))
    check_gates(s4, x, 1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fast", [-4.0, -8.0, -12.0, -16.0, -40.0, -70.0])
def test_tokens_that_forget_among_others(s4, dtype, fast):  # noqa: F811
    """Tokens that nearly reset the state among slow ones: at the ends of chunks and segments, alone, next
    to each other, and as whole chunks."""
    T = 700
    x = inputs(7, 2 * T, 2, 1, 4, 16, 24, dtype)
    x["g"] = -0.02 * uniform(1, 2 * T, 4)
    for h, places in enumerate([[0, 63, 64, 127, 128, 300, 400, 401, 699], [100], list(range(192, 260)), []]):
        for t in places:
            x["g"][t, h] = fast
            x["g"][T + (t + 31) % T, h] = 1.1 * fast
    check_gates(s4, x, 2)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("gates", ["token", "head"])
@pytest.mark.parametrize("offsets", [[0, 0, 1, 65, 65, 200], [3, 20, 20, 130, 131, 190], [0, 300, 300, 301, 900, 1000],
                                     [1, 258, 516, 774, 1032, 1289], [0, 0, 0, 0, 0, 0]])
def test_packed_gates(s4, dtype, gates, offsets):  # noqa: F811
    x = inputs(offsets[-1] + 1, offsets[-1] + 5, 5, 1, 3, 24, 40, dtype, gates=gates)
    x["g"] = x["g"] * torch.tensor([0.1, 1.0, 12.0])
    check_gates(s4, x, 5, offsets)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("T,dk,dv", [(100, 256, 256), (300, 72, 200), (90, 200, 129), (400, 130, 33)])
def test_large_heads(s4, dtype, T, dk, dv):  # noqa: F811
    x = inputs(T, T, 1, 2, 2, dk, dv, dtype)
    x["g"] = x["g"] * torch.tensor([0.2, 10.0])
    check_gates(s4, x, 1)


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("T", [1, 2, 64, 65, 300])
def test_gates_of_resets(s4, T, state):  # noqa: F811
    """g = -infinity: its dg is 0, and its neighbours have theirs."""
    x = inputs(T, T, 1, 2, 2, 16, 16, F32, state=state)
    x["g"][T // 2, 0], x["g"][T - 1, 1], x["g"][0, 1] = -math.inf, -1e30, -math.inf
    check_gates(s4, x, 1)


def test_wide_range_of_values(s4):  # noqa: F811
    """Tokens whose values are a thousand times the others' leave the others' dg its digits."""
    x = inputs(2, 300, 1, 2, 2, 16, 16, F32)
    x["g"] = torch.where(uniform(3, 300, 2) < 0.1, -9.0, -0.3)
    for t in (10, 70, 130, 200):
        x["v"][t] *= 1000
        x["dout"][t + 5] *= 1000
    check_gates(s4, x, 1)
