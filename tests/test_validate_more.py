"""CPU tests of S4DPLR_VALIDATE=1 for linear attention, the root-mean-square norm, quantization and
the 8-bit product: the checks come before anything else, so CPU tensors reach them; what passes
them is refused for being no GPU tensor."""
import math

import pytest
import torch

T, S, H, K, V = 10, 2, 1, 4, 3
NAN, INF = math.nan, math.inf


@pytest.fixture
def s4(monkeypatch):
    import structured_state_space_dplr_amd as s4
    monkeypatch.setenv("S4DPLR_VALIDATE", "1")
    return s4


def inputs():
    x = {n: torch.ones(T, H, K if n in "qk" else V) for n in ("q", "k", "v", "dout")}
    x.update(g=-torch.ones(T, H))
    x.update({n: torch.zeros(S, H, K, V) for n in ("state", "dstate_out")})
    return x


def call(s4, x, offsets=None, bwd=False):
    plan = s4.LinearAttentionPlan(S, T, H, H, K, V, torch.float32, training=True)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    head = (plan, x["q"], x["k"], x["v"], x["g"])
    if bwd:
        s4.linear_attention_bwd(*head, None, x["dout"], x["dstate_out"], *[None] * 5, None, offsets=off)
    else:
        s4.linear_attention_fwd(*head, x["state"], None, None, None, offsets=off)


def refused(s4, match, *args, **kw):
    with pytest.raises(ValueError, match=match) as e:
        call(s4, *args, **kw)
    assert isinstance(e.value, s4.S4DPLRPreconditionError) == (match != "GPU tensor")


@pytest.mark.parametrize("bwd", [False, True])
def test_valid_calls_pass(s4, bwd):
    x = inputs()
    x["g"][3] = -INF                                 # a reset
    for offsets in (None, [0, 5, 10], [2, 2, 7], [0, 0, 0], [10, 10, 10]):
        refused(s4, "GPU tensor", x, offsets, bwd=bwd)
    for g in (None, -torch.ones(H), torch.zeros(H)):
        refused(s4, "GPU tensor", dict(x, g=g), bwd=bwd)


@pytest.mark.parametrize("bwd", [False, True])
def test_bad_values(s4, bwd):
    for n in ("q", "k", "v", "g", "dout" if bwd else "state", *(["dstate_out"] if bwd else [])):
        for bad in (NAN, INF):
            x = inputs()
            x[n].view(-1)[2] = bad
            refused(s4, n if n != "g" else "g must be", x, bwd=bwd)
    refused(s4, "g must be", dict(inputs(), g=torch.full((H,), 0.5)), bwd=bwd)
    for offsets in ([-1, 5, 10], [0, 6, 5], [0, 5, 11]):
        refused(s4, "offsets", inputs(), offsets, bwd=bwd)


def test_rows_outside_may_hold_anything(s4):
    x = inputs()
    for n in ("q", "k", "v", "g"):
        x[n][:2], x[n][8:] = NAN, INF
    refused(s4, "GPU tensor", x, [2, 5, 8])


def test_the_others(s4):
    x, bad = torch.ones(4, 256), torch.ones(4, 256)
    bad[1, 7] = NAN
    q = torch.ones(4, 256).to(torch.float8_e4m3fn)
    sc = torch.full((4, 2), 127, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    nan = torch.full((4, 2), 255, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    rstd, gamma, out = torch.ones(4), torch.ones(256), torch.ones(4, 4)
    error = s4.S4DPLRPreconditionError
    for fn, args in ((s4.rms_norm_fwd, (bad, None, gamma, None, x)), (s4.rms_norm_fwd, (x, bad, gamma, None, x)),
                     (s4.rms_norm_bwd, (x, gamma, rstd, bad, None, None, None, None)),
                     (s4.rms_norm_bwd, (x, gamma, rstd, x, bad, None, None, None))):
        with pytest.raises(error, match="not finite"):
            fn(*args)
    # matrices are looked at by shape and place first
    for fn, args in ((s4.quantize_fp8, (bad, q, sc)), (s4.matmul_fp8, (q, nan, q, sc, out))):
        with pytest.raises(ValueError, match="GPU tensor"):
            fn(*args)
