"""GPU tests of the gated delta rule's workspace: packed batches that put as many chunks as
their plan can hold into it, and what lies behind it."""
import pytest
import torch

from test_gpu_delta import BF, F32, check_backward, check_forward, close, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def packed(lengths, first=0):
    return [first] + (torch.tensor(lengths).cumsum(0) + first).tolist()


# 2 value heads of 16: up to 8 tokens go token by token, 16 from 129 sequences on
SHORT = [[9] * 12 + [0] * 20 + [1] * 12, [9, 0] * 40, [0] * 30 + [200] + [0] * 30 + [9, 8, 10] + [1] * 20,
         [8] * 5 + [9] * 5 + [0] * 10, [64, 0, 0, 0, 0, 0, 0, 0, 65] + [0] * 20 + [9],
         [0] * 300 + [17] * 100, ([16] * 3 + [17] + [0]) * 40, [1] * 150 + [700] + [0] * 60]


@pytest.mark.parametrize("i", range(len(SHORT)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_short_and_long(s4, i, dtype):
    lengths = SHORT[i]
    offsets = packed(lengths, i % 3)
    check_forward(s4, inputs(i, offsets[-1] + i % 2, len(lengths), 1, 2, 16, 16, dtype), len(lengths), offsets)


@pytest.mark.parametrize("i", [0, 2, 4])
def test_gradients_of_packed_short_and_long(s4, i):
    lengths = SHORT[i]
    offsets = packed(lengths, 1)
    check_backward(s4, inputs(i, offsets[-1] + 3, len(lengths), 1, 2, 16, 16, BF), len(lengths), offsets)


@pytest.mark.parametrize("lengths,training", [([9] * 12 + [0] * 20, False), ([1] * 40, False), ([1] * 8, False),
                                              ([9] * 12 + [0] * 20, True), ([130], True)])
def test_nothing_is_written_behind_the_workspace(s4, lengths, training):
    S, T = len(lengths), sum(lengths)
    x = inputs(S, T, S, 1, 2, 16, 16, BF)
    d = {n: t.cuda() for n, t in x.items()}
    p = s4.DeltaPlan(S, T, 1, 2, 16, 16, BF, training=training)
    room = 1 << 16
    guarded = lambda n: torch.full((n + 2 * room,), 0x5a, dtype=torch.uint8, device="cuda")  # noqa: E731
    ws, saved = guarded(p.workspace_bytes), guarded(p.saved_bytes)
    inner = lambda t: t[room:-room]  # noqa: E731
    o, new = torch.empty_like(d["v"]), torch.empty_like(d["state"])
    off = torch.tensor(packed(lengths), dtype=torch.int32, device="cuda")
    s4.delta_fwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], o, new, inner(ws),
                 saved=inner(saved) if training else None, scale=0.7, offsets=off)
    if training:
        g = [torch.empty_like(d[n]) for n in ("q", "k", "v", "g", "beta", "state")]
        s4.delta_bwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], inner(saved), d["dout"],
                     d["dstate_out"], *g, inner(ws), scale=0.7, offsets=off)
    for t in (ws, saved):
        assert bool((t[:room] == 0x5a).all()) and bool((t[-room:] == 0x5a).all())
    z = {n: t.double() for n, t in x.items()}
    bounds = list(zip(packed(lengths)[:-1], packed(lengths)[1:]))
    ro, rs = reference(z["q"], z["k"], z["v"], z["g"], z["beta"], z["state"], 0.7, bounds)
    close(o, ro, "o")
    close(new, rs, "state")
