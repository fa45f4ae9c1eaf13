"""CPU tests of S4DPLR_VALIDATE=1 for the token-major operators: the checks come before
anything else, so CPU tensors reach them; what passes them is refused for being no GPU
tensor."""
import math

import pytest
import torch


@pytest.fixture
def s4(monkeypatch):
    import structured_state_space_dplr_amd as s4
    monkeypatch.setenv("S4DPLR_VALIDATE", "1")
    return s4


T, S, H, K, V = 10, 2, 1, 4, 3
NAN, INF = math.nan, math.inf


def delta_inputs():
    x = {n: torch.ones(T, H, K if n in "qk" else V) for n in ("q", "k", "v", "dout")}
    x.update(g=-torch.ones(T, H), beta=torch.ones(T, H))
    x.update({n: torch.zeros(S, H, K, V) for n in ("state", "dstate_out")})
    return x


def call(s4, x, offsets=None, bwd=False):
    plan = s4.DeltaPlan(S, T, H, H, K, V, torch.float32, training=True)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    head = (plan, x["q"], x["k"], x["v"], x["g"], x["beta"])
    if bwd:
        s4.delta_bwd(*head, None, x["dout"], x["dstate_out"], *[None] * 6, None, offsets=off)
    else:
        s4.delta_fwd(*head, x["state"], None, None, None, offsets=off)


def refused(s4, match, *args, **kw):
    with pytest.raises(ValueError, match=match) as e:
        call(s4, *args, **kw)
    assert isinstance(e.value, s4.S4DPLRPreconditionError) == (match != "GPU tensor")


@pytest.mark.parametrize("bwd", [False, True])
def test_valid_calls_pass(s4, bwd):
    x = delta_inputs()
    x["g"][3] = -INF                                 # a reset
    for offsets in (None, [0, 5, 10], [2, 2, 7], [0, 0, 0], [10, 10, 10]):
        refused(s4, "GPU tensor", x, offsets, bwd=bwd)


@pytest.mark.parametrize("offsets", [[-1, 5, 10], [0, 6, 5], [0, 5, 11], [11, 11, 11],
                                     [-2 ** 31, 0, 10], [0, 2 ** 31 - 1, 10], [5, 0, 10]])
@pytest.mark.parametrize("bwd", [False, True])
def test_offsets_that_do_not_rise_within_the_rows(s4, offsets, bwd):
    refused(s4, "offsets", delta_inputs(), offsets, bwd=bwd)


@pytest.mark.parametrize("offsets", [[], [0], [0, 5, 10, 10]])
def test_offsets_of_another_length(s4, offsets):
    refused(s4, "GPU tensor", delta_inputs(), offsets)      # the tensors' own checks come next


@pytest.mark.parametrize("name,bwd", [("q", 0), ("k", 0), ("v", 0), ("beta", 0), ("state", 0),
                                      ("q", 1), ("v", 1), ("dout", 1), ("dstate_out", 1)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_values_that_are_not_finite(s4, name, bwd, value):
    x = delta_inputs()
    x[name].view(x[name].shape[0], -1)[1, -1] = value
    refused(s4, name + " is not finite", x, bwd=bool(bwd))


@pytest.mark.parametrize("value", [NAN, INF, 0.5])
def test_log_decays(s4, value):
    x = delta_inputs()
    x["g"][4] = value
    refused(s4, "g must be <= 0", x)


@pytest.mark.parametrize("bwd", [False, True])
def test_rows_outside_the_sequences_may_hold_anything(s4, bwd):
    x = delta_inputs()
    for n in ("q", "k", "v", "g", "beta", "dout"):
        x[n][:2] = x[n][8:] = NAN
    refused(s4, "GPU tensor", x, [2, 4, 8], bwd=bwd)
    refused(s4, "is not finite", x, [1, 4, 8], bwd=bwd)
    refused(s4, "is not finite", x, [2, 4, 9], bwd=bwd)


@pytest.mark.parametrize("name", ["x", "gamma", "mean", "rstd", "dy"])
def test_norm_gradients(s4, name):
    a = {"x": torch.ones(3, 5), "gamma": torch.ones(5), "mean": torch.ones(3),
         "rstd": torch.ones(3), "dy": torch.ones(3, 5)}
    a[name].view(-1)[-1] = NAN
    with pytest.raises(s4.S4DPLRPreconditionError, match=name + " is not finite"):
        s4.layer_norm_bwd(*a.values(), None, None, None, None)
