"""GPU tests of the gradient of linear attention's decays, dg: every set of outputs, on a workspace
that holds nothing of an earlier call."""
import itertools

import pytest
import torch

from test_gpu_linear_attention import BF, F16, F32, backward, forward, inputs, s4  # noqa: F401

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
