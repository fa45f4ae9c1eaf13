"""GPU tests of how many bits the gated delta rule carries with tensors of 16 bits.

A value of 16 bits is one value of 32, and everything behind the loads is defined
in 32 bits: a call in bf16 or fp16 and the call in fp32 on the same values differ
in the rounding of the 16-bit outputs alone, and states, dg and dbeta are equal.
(The parts that an fp32 operand has beyond a 16-bit one are zero, and adding their
products changes no sum.)  So these comparisons have no tolerance.

Keys and queries that share a direction make the pairs' products large, and values
that nearly cancel show what an operand of too few bits loses."""
import pytest
import torch

from test_gpu_delta import backward, check_backward, check_forward, forward, inputs, reference

pytestmark = pytest.mark.gpu

BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def related(seed, tokens, S, Hk, Hv, dk, dv, dtype, share):
    """``inputs`` with weak decay and unit keys and queries of which all have
    ``share`` of one direction."""
    x = inputs(seed, tokens, S, Hk, Hv, dk, dv, torch.float64)
    line = torch.full((dk,), dk ** -0.5, dtype=torch.float64)
    for n in ("q", "k"):
        t = share * line + (1 - share * share) ** 0.5 * x[n]
        x[n] = t / t.norm(dim=-1, keepdim=True)
    for n in ("q", "k", "v", "dout"):
        x[n] = x[n].to(dtype)
    x["g"] *= 0.1
    return x


def widened(x):
    return {n: None if t is None else t.float() for n, t in x.items()}


SIZES = [(1, 5, 2, 2, 64, 48), (2, 200, 2, 2, 64, 48), (1, 300, 1, 3, 128, 64),
         (1, 130, 1, 1, 200, 40), (5, 130, 6, 18, 128, 128)]


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("S,T,Hk,Hv,dk,dv", SIZES)
@pytest.mark.parametrize("training", [False, True])
def test_16_bit_tensors_give_the_fp32_outputs(s4, dtype, S, T, Hk, Hv, dk, dv, training):
    x = related(T + dk, S * T, S, Hk, Hv, dk, dv, dtype, 0.8)
    o, new = forward(s4, x, S, training=training)[4:]
    wo, wnew = forward(s4, widened(x), S, training=training)[4:]
    assert torch.equal(new, wnew), "state"
    assert torch.equal(o, wo.to(dtype)), f"o: {(o != wo.to(dtype)).double().mean():.1e} differ"


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("S,T,Hk,Hv,dk,dv", SIZES)
def test_16_bit_tensors_give_the_fp32_gradients(s4, dtype, S, T, Hk, Hv, dk, dv):
    x = related(T + dk, S * T, S, Hk, Hv, dk, dv, dtype, 0.8)
    got, want = backward(s4, x, S)[2], backward(s4, widened(x), S)[2]
    for n in ("state", "g", "beta"):
        assert torch.equal(got[n], want[n]), "d" + n
    for n in ("q", "k", "v"):
        assert torch.equal(got[n], want[n].to(dtype)), "d" + n


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("share", [0.9, 1.0])
def test_related_keys_and_queries(s4, dtype, share):
    x = related(1, 200, 1, 1, 2, 32, 24, dtype, share)
    check_forward(s4, x, 1)
    check_backward(s4, x, 1)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_values_that_cancel(s4, dtype):
    """Two orthogonal keys write b0 v and -b1 v with 3 b0 = 2 b1 (1 + 2^-12); a query (3 m, 2 m)
    reads m v 2 b1 2^-12, a difference of two terms 2^12 times as large.  fp32 sums lose
    at most 8 half steps of the terms, 2^-9 of the result, and the output's rounding is
    2^-8 (bf16) or 2^-11 of it; a term held in 17 bits is off by up to 2^-18, 2^-6 of the result."""
    T, dv = 64, 64
    gen = torch.Generator().manual_seed(5)
    x = {n: torch.zeros(T, 1, 16) for n in ("q", "k")}
    x["k"][0, 0, 0] = x["k"][1, 0, 1] = 1
    m = torch.randint(16, 32, (T,), generator=gen) / 64.0
    x["q"][2:, 0, 0], x["q"][2:, 0, 1] = 3 * m[2:], 2 * m[2:]
    v = torch.randn(1, dv, generator=gen).to(dtype).float()
    x["v"] = torch.zeros(T, 1, dv)
    x["v"][0], x["v"][1] = v, -v
    x = {n: t.to(dtype) for n, t in x.items()}
    x["g"], x["beta"] = torch.zeros(T, 1), torch.zeros(T, 1)
    x["beta"][1] = 0.9137
    x["beta"][0] = (x["beta"][1].double() * (2 + 2.0 ** -11) / 3).float()
    x.update(state=None)
    o = forward(s4, x, 1)[4].double().cpu()[2:]
    z = {n: x[n].double() for n in ("q", "k", "v", "g", "beta")}
    want = reference(*z.values(), torch.zeros(1, 1, 16, dv, dtype=torch.float64), 0.7, [(0, T)])[0][2:]
    term = 0.7 * (z["q"][2:, :, :1] * z["beta"][0] * z["v"][0].abs())
    lim = torch.finfo(dtype).eps / 2 * want.abs() + 8 * 2.0 ** -24 * term
    if dtype == F16:
        lim = lim + 2.0 ** -25
    assert bool(((o - want).abs() <= lim).all()), float(((o - want).abs() / lim).max())
