"""GPU tests of the gated delta rule (delta_fwd, delta_bwd) against the
recurrence token by token in 64 bits, its reverse-mode gradients and central
differences.

Tolerances: an output of b bits is rounded once (half a step: eps / 2 of the
value).  Before that, every value is a chain of fp32 sums of at most
dk + 2 * 64 terms per chunk, whose rounding errors (2^-24 of the largest term
each, independent of each other) add up as the square root of their number: at
most sqrt(384) < 20 per sum, three sums after one another per chunk, and what a
chunk adds to the state fades like the state itself.  64 * 2^-24 of the largest
value of the output allows for that; dg and dbeta, sums over rows of such
products, get four times it."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def reference(q, k, v, g, beta, state, scale, bounds):
    """o [tokens, Hv, dv] and the last states, in 64 bits; bounds: (start, end) per sequence."""
    Hk, Hv = q.shape[1], v.shape[1]
    heads = torch.arange(Hv) // (Hv // Hk)
    rows, last = {}, []
    for s, (a, b) in enumerate(bounds):
        S = state[s]
        for t in range(a, b):
            S = S * g[t].exp()[:, None, None]
            kt, qt = k[t][heads], q[t][heads]
            n = v[t] - (S * kt[:, :, None]).sum(1)
            S = S + kt[:, :, None] * (beta[t][:, None] * n)[:, None, :]
            rows[t] = scale * (S * qt[:, :, None]).sum(1)
        last.append(S)
    zero = torch.zeros(Hv, v.shape[2], dtype=torch.float64)
    o = torch.stack([rows.get(t, zero) for t in range(q.shape[0])]) if q.shape[0] else v.clone()
    return o, torch.stack(last)


def inputs(seed, tokens, S, Hk, Hv, dk, dv, dtype, state=True):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda t: t / (t.norm(dim=-1, keepdim=True) + 1e-6)  # noqa: E731
    x = {"q": unit(rnd(tokens, Hk, dk)), "k": unit(rnd(tokens, Hk, dk)), "v": rnd(tokens, Hv, dv)}
    x = {n: t.to(dtype) for n, t in x.items()}
    x["g"] = (-torch.nn.functional.softplus(rnd(tokens, Hv) - 2)).float()
    x["beta"] = torch.sigmoid(rnd(tokens, Hv)).float()
    x["state"] = 0.3 * rnd(S, Hv, dk, dv).float() if state else None
    x["dout"] = rnd(tokens, Hv, dv).to(dtype)
    x["dstate_out"] = 0.3 * rnd(S, Hv, dk, dv).float()
    return x


def bounds_of(S, tokens, offsets):
    if offsets is None:
        n = tokens // S
        return [(i * n, i * n + n) for i in range(S)]
    return list(zip(offsets[:-1], offsets[1:]))


def close(got, ref, name, factor=1.0):
    assert got.shape == ref.shape, name
    if ref.numel() == 0:
        return
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    err = (got.double().cpu() - ref).abs()
    lim = half * ref.abs() + factor * 64 * UNIT * max(float(ref.abs().max()), 1e-30)
    if got.dtype == torch.float16:
        lim = lim + 2.0 ** -25          # half a step of its smallest numbers
    worst = float((err / lim).max())
    assert worst <= 1, f"{name}: {worst:.2f} of the tolerance"


def forward(s4, x, S, offsets=None, training=False, scale=0.7, in_place=False, plan=None):
    tokens, Hk, dk = x["q"].shape
    Hv, dv = x["v"].shape[1:]
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    p = plan or s4.DeltaPlan(S, tokens, Hk, Hv, dk, dv, x["v"].dtype, training=training)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o = torch.full((tokens, Hv, dv), 7.0, dtype=x["v"].dtype, device="cuda")
    new = d["state"] if in_place else torch.full((S, Hv, dk, dv), 7.0, device="cuda")
    saved = p.saved() if training else None
    s4.delta_fwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], o, new, p.workspace(),
                 saved=saved, scale=scale, offsets=off)
    return p, d, off, saved, o, new


def check_forward(s4, x, S, offsets=None, **kw):
    tokens = x["q"].shape[0]
    _, _, _, _, o, new = forward(s4, x, S, offsets, **kw)
    z = {n: None if t is None else t.double() for n, t in x.items()}
    if z["state"] is None:
        z["state"] = torch.zeros(S, x["v"].shape[1], x["q"].shape[2], x["v"].shape[2],
                                 dtype=torch.float64)
    bounds = bounds_of(S, tokens, offsets)
    ro, rs = reference(z["q"], z["k"], z["v"], z["g"], z["beta"], z["state"], 0.7, bounds)
    inside = torch.zeros(tokens, dtype=torch.bool)
    for a, b in bounds:
        inside[a:b] = True
    close(o[inside.cuda()], ro[inside], "o")
    close(new, rs, "state")
    assert bool((o[~inside.cuda()] == 7.0).all()), "rows outside every sequence were written"


BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 63, 64, 65, 150])
def test_lengths(s4, dtype, T):
    check_forward(s4, inputs(T, 2 * T, 2, 2, 2, 32, 16, dtype), 2)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (40, 72), (64, 17), (65, 16), (128, 128),
                                   (129, 33), (256, 256)])
@pytest.mark.parametrize("T", [3, 70])
def test_head_sizes(s4, dtype, dk, dv, T):
    check_forward(s4, inputs(dk * 7 + dv, T, 1, 1, 2, dk, dv, dtype), 1)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 5), (3, 3), (2, 6)])
@pytest.mark.parametrize("T", [5, 100])
def test_head_groups(s4, Hk, Hv, T):
    check_forward(s4, inputs(Hv, 3 * T, 3, Hk, Hv, 24, 40, BF), 3)


@pytest.mark.parametrize("offsets", [
    [0, 0, 1, 65, 65, 200], [3, 20, 20, 130, 131, 190], [0, 200, 200, 200, 200, 200],
    [0, 0, 0, 0, 0, 0], [0, 16, 33, 34, 97, 161]])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("state", [True, False])
def test_packed_sequences(s4, offsets, dtype, state):
    # empty and one-token sequences, rows before the first and behind the last one
    check_forward(s4, inputs(9, 200, 5, 1, 2, 32, 24, dtype, state=state), 5, offsets)


@pytest.mark.parametrize("dk,dv", [(128, 128), (100, 120), (65, 33), (128, 17)])
def test_many_heads(s4, dk, dv):
    # more slices of 16 columns than the GPU has CUs: the blocks take 32
    x = inputs(dk + dv, 5 * 130, 5, 6, 18, dk, dv, BF)
    check_forward(s4, x, 5)
    check_backward(s4, x, 5)


def test_many_heads_packed(s4):
    x = inputs(77, 300, 6, 16, 16, 128, 48, BF)
    offsets = [2, 2, 3, 131, 200, 264, 290]
    check_forward(s4, x, 6, offsets)
    check_backward(s4, x, 6, offsets)


@pytest.mark.parametrize("offsets", [[0, 1, 2, 2, 5, 12], [0, 1, 41, 41, 42, 45], [0, 3, 6, 8, 9, 9]])
def test_packed_short_sequences(s4, offsets):
    # token by token, token by token beside chunks, token by token with an empty one
    check_forward(s4, inputs(19, offsets[-1], 5, 1, 2, 32, 24, BF), 5, offsets)
    x = inputs(20, offsets[-1], 5, 8, 8, 32, 112, F32)
    check_forward(s4, x, 5, offsets)


def test_many_sequences(s4):
    # more sequences than a wave has lanes
    gen = torch.Generator().manual_seed(0)
    offsets = [0] + torch.randint(0, 4, (150,), generator=gen).cumsum(0).tolist()
    offsets[-1] += 70
    check_forward(s4, inputs(1, offsets[-1] + 3, 150, 1, 1, 16, 16, BF), 150, offsets)


@pytest.mark.parametrize("S", [65, 4097])
def test_thousands_of_packed_sequences(s4, S):
    # three of them are longer than a chunk, a third is empty
    gen = torch.Generator().manual_seed(S)
    lengths = torch.randint(0, 3, (S,), generator=gen)
    lengths[torch.tensor([0, S // 2, S - 1])] = torch.tensor([70, 130, 65])
    offsets = [0] + torch.cumsum(lengths, 0).tolist()
    x = inputs(S, offsets[-1], S, 1, 1, 8, 8, F32)
    check_forward(s4, x, S, offsets)
    check_backward(s4, x, S, offsets)


@pytest.mark.parametrize("T", [8, 130])
@pytest.mark.parametrize("reset", [-math.inf, torch.finfo(torch.float32).min, -1e4, -150.0, -60.0])
def test_resets(s4, reset, T):
    # a token that forgets everything, in the middle and at the start of chunks; what
    # follows must not lose digits to the large number
    x = inputs(4, T, 1, 1, 2, 32, 16, F32)
    x["g"][[0, 3, T // 2, T - 2], 0] = reset
    if T > 64:
        x["g"][64, 1] = reset
    check_forward(s4, x, 1)


@pytest.mark.parametrize("T", [8, 130])
def test_masked_tokens(s4, T):
    # beta = 0: nothing is written; zero keys, queries and values; no decay
    x = inputs(5, T, 1, 2, 2, 32, 16, BF)
    x["beta"][::3] = 0
    x["k"][1::4] = 0
    x["q"][2::5] = 0
    x["v"][3::7] = 0
    x["g"][::2] = 0
    x["beta"][1::6] = 1
    check_forward(s4, x, 1)


def test_equal_keys(s4):
    # the inverse's entries stay bounded, products of its powers would not
    x = inputs(6, 128, 1, 1, 1, 32, 16, F32)
    x["k"][:] = x["k"][0]
    x["beta"][:] = 1
    x["g"][:] = 0
    check_forward(s4, x, 1)


def test_whole_batch_masked(s4):
    x = inputs(7, 70, 1, 1, 1, 16, 16, BF)
    x["beta"][:] = 0
    check_forward(s4, x, 1)


@pytest.mark.parametrize("cut", [[1] * 9, [70, 1, 1, 64, 5], [64, 64], [17, 200]])
def test_stream_in_pieces(s4, cut):
    """Consecutive calls that carry the state in place continue one sequence."""
    T = sum(cut)
    x = inputs(8, T, 1, 1, 2, 32, 24, F32)
    z = {n: t.double() for n, t in x.items()}
    ro, rs = reference(z["q"], z["k"], z["v"], z["g"], z["beta"], z["state"], 0.7, [(0, T)])
    state, at, outs = x["state"].cuda(), 0, []
    for n in cut:
        piece = {m: x[m][at:at + n] for m in ("q", "k", "v", "g", "beta", "dout")}
        piece["state"] = state
        outs.append(forward(s4, piece, 1, in_place=True)[4])
        at += n
    close(torch.cat(outs), ro, "o")
    close(state, rs, "state")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [4, 80])
@pytest.mark.parametrize("shift", [0, 1])
def test_columns_of_one_matrix(s4, dtype, T, shift):
    # q, k, v as column ranges of a projection's output, at odd widths and addresses
    Hk, Hv, dk, dv = 2, 2, 24, 21
    x = inputs(10, T, 1, Hk, Hv, dk, dv, dtype)
    wide = torch.zeros(T * (2 * Hk * dk + Hv * dv + 3) + shift, dtype=dtype, device="cuda")
    m = wide[shift:].view(T, -1)
    views = {}
    for n, c in (("q", 1), ("k", 1 + Hk * dk), ("v", 2 + 2 * Hk * dk)):
        H, d = x[n].shape[1:]
        views[n] = m[:, c:c + H * d].unflatten(1, (H, d))
        views[n].copy_(x[n])
    p = s4.DeltaPlan(1, T, Hk, Hv, dk, dv, dtype)
    got = []
    for src in (views, {n: x[n].cuda() for n in views}):
        o = torch.empty(T, Hv, dv, dtype=dtype, device="cuda")
        new = torch.empty(1, Hv, dk, dv, device="cuda")
        s4.delta_fwd(p, src["q"], src["k"], src["v"], x["g"].cuda(), x["beta"].cuda(),
                     x["state"].cuda(), o, new, p.workspace())
        got.append((o, new))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def backward(s4, x, S, offsets=None, skip=(), scale=0.7, use_dstate=True):
    p, d, off, saved, o, new = forward(s4, x, S, offsets, training=True, scale=scale)
    g = {n: torch.full_like(d[n], 7.0) for n in ("q", "k", "v", "g", "beta")}
    g["state"] = torch.full_like(d["dstate_out"], 7.0)
    g = {n: None if n in skip else t for n, t in g.items()}
    s4.delta_bwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], saved, d["dout"],
                 d["dstate_out"] if use_dstate else None, g["q"], g["k"], g["v"], g["g"],
                 g["beta"], g["state"], p.workspace(), scale=scale, offsets=off)
    return o, new, g


def reference_grads(x, S, offsets, use_dstate=True, scale=0.7):
    tokens = x["q"].shape[0]
    names = ("q", "k", "v", "g", "beta", "state")
    z = {n: None if x[n] is None else x[n].double() for n in names}
    if z["state"] is None:
        z["state"] = torch.zeros_like(x["dstate_out"], dtype=torch.float64)
    leaves = {n: z[n].requires_grad_() for n in names}
    o, last = reference(*(leaves[n] for n in names), scale, bounds_of(S, tokens, offsets))
    loss = (o * x["dout"].double()).sum() + 0 * leaves["state"].sum()
    if use_dstate:
        loss = loss + (last * x["dstate_out"].double()).sum()
    grads = torch.autograd.grad(loss, [leaves[n] for n in names], allow_unused=True)
    return {n: torch.zeros_like(z[n]) if t is None else t for n, t in zip(names, grads)}


def check_backward(s4, x, S, offsets=None, use_dstate=True):
    _, _, got = backward(s4, x, S, offsets, use_dstate=use_dstate)
    ref = reference_grads(x, S, offsets, use_dstate)
    inside = torch.zeros(x["q"].shape[0], dtype=torch.bool)
    for a, b in bounds_of(S, x["q"].shape[0], offsets):
        inside[a:b] = True
    for n in ("q", "k", "v", "g", "beta"):
        close(got[n][inside.cuda()], ref[n][inside], "d" + n, 4.0 if n in ("g", "beta") else 1.0)
        assert bool((got[n][~inside.cuda()] == 7.0).all()), n
    close(got["state"], ref["state"], "dstate")


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 150])
def test_gradients_lengths(s4, dtype, T):
    check_backward(s4, inputs(T, 2 * T, 2, 2, 2, 32, 16, dtype), 2)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (40, 72), (64, 17), (65, 16), (128, 128),
                                   (129, 33), (256, 256)])
def test_gradients_head_sizes(s4, dtype, dk, dv):
    check_backward(s4, inputs(dk * 7 + dv, 70, 1, 1, 2, dk, dv, dtype), 1)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 5), (3, 3), (2, 6)])
def test_gradients_head_groups(s4, Hk, Hv):
    check_backward(s4, inputs(Hv, 3 * 70, 3, Hk, Hv, 24, 40, BF), 3)


@pytest.mark.parametrize("offsets", [
    [0, 0, 1, 65, 65, 200], [3, 20, 20, 130, 131, 190], [0, 0, 0, 0, 0, 0]])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("state", [True, False])
def test_gradients_packed(s4, offsets, dtype, state):
    check_backward(s4, inputs(9, 200, 5, 1, 2, 32, 24, dtype, state=state), 5, offsets,
                   use_dstate=state)


@pytest.mark.parametrize("reset", [-math.inf, -1e4, -60.0])
def test_gradients_resets(s4, reset):
    x = inputs(4, 130, 1, 1, 2, 32, 16, F32)
    x["g"][[0, 3, 65, 128], 0] = reset
    x["g"][64, 1] = reset
    check_backward(s4, x, 1)


def test_gradients_masked_tokens(s4):
    x = inputs(5, 130, 1, 2, 2, 32, 16, F32)
    x["beta"][::3] = 0
    x["k"][1::4] = 0
    x["q"][2::5] = 0
    x["v"][3::7] = 0
    x["g"][::2] = 0
    x["dout"][5::9] = 0
    check_backward(s4, x, 1)


def test_gradients_against_differences(s4):
    """<gradient, direction> against central differences of the 64-bit loss.  The
    difference with step h is off by about h^2 |f'''| / 6 + 2^-53 |f| / h: under
    1e-8 of f at h = 1e-4 for a loss that is smooth at scale 1; the gradient's own
    error is that of ``close``, summed over up to 5000 terms of random signs."""
    x = inputs(12, 90, 1, 1, 2, 16, 12, F32)
    _, _, got = backward(s4, x, 1)
    gen = torch.Generator().manual_seed(3)
    names = ("q", "k", "v", "g", "beta", "state")
    for n in names:
        e = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        loss = []
        for h in (1e-4, -1e-4):
            z = {m: x[m].double() + (h * e if m == n else 0) for m in names}
            o, last = reference(*(z[m] for m in names), 0.7, [(0, 90)])
            loss.append((o * x["dout"].double()).sum() + (last * x["dstate_out"].double()).sum())
        slope = float(loss[0] - loss[1]) / 2e-4
        mine = float((got[n].double().cpu() * e).sum())
        size = float((got[n].double().cpu() * e).abs().sum())
        assert abs(mine - slope) <= 1e-5 * size, (n, mine, slope)


@pytest.mark.parametrize("skip", [("q",), ("k", "v"), ("g", "beta"), ("state",),
                                  ("q", "k", "g", "beta")])
def test_gradients_left_out(s4, skip):
    x = inputs(13, 70, 1, 1, 2, 24, 20, BF)
    _, _, full = backward(s4, x, 1)
    _, _, some = backward(s4, x, 1, skip=skip)
    for n, t in some.items():
        assert (t is None) == (n in skip)
        if t is not None:
            assert torch.equal(t, full[n]), n


def test_equal_calls_give_equal_bits(s4):
    x = inputs(14, 300, 2, 1, 4, 64, 48, BF)
    a, b = backward(s4, x, 2), backward(s4, x, 2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for n in a[2]:
        assert torch.equal(a[2][n], b[2][n]), n


@pytest.mark.parametrize("T", [4, 200])
def test_no_state_wanted(s4, T):
    x = inputs(15, T, 1, 1, 1, 16, 16, BF)
    d = {n: t.cuda() for n, t in x.items()}
    p = s4.DeltaPlan(1, T, 1, 1, 16, 16, BF)
    o = [torch.empty_like(d["v"]) for _ in range(2)]
    new = torch.empty_like(d["state"])
    for i in range(2):
        s4.delta_fwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], o[i],
                     new if i else None, p.workspace())
    assert torch.equal(o[0], o[1])


@pytest.mark.parametrize("T", [1, 100])
def test_graph_replays(s4, T):
    """Forward and (T > 1) backward captured once, replayed with eager work in
    between and new inputs in the same buffers."""
    train = T > 1
    x = inputs(16, 2 * T, 2, 1, 2, 32, 32, BF)
    p, d, _, saved, o, new = forward(s4, x, 2, training=train)
    g = {n: torch.empty_like(d[n]) for n in ("q", "k", "v", "g", "beta")}
    gs, ws = torch.empty_like(new), p.workspace()

    def call():
        s4.delta_fwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], o, new, ws,
                     saved=saved, scale=0.7)
        if train:
            s4.delta_bwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], saved, d["dout"],
                         d["dstate_out"], g["q"], g["k"], g["v"], g["g"], g["beta"], gs, ws,
                         scale=0.7)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    outs = [o, new] + ([gs, *g.values()] if train else [])
    for i in range(4):
        y = inputs(20 + i, 2 * T, 2, 1, 2, 32, 32, BF)
        for n in d:
            d[n].copy_(y[n])
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i


def test_two_streams_with_their_own_workspaces(s4):
    x = [inputs(30 + i, 400, 2, 1, 2, 64, 64, BF) for i in range(2)]
    want = [backward(s4, y, 2) for y in x]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for st, y in zip(streams, x):
        with torch.cuda.stream(st):
            got.append(backward(s4, y, 2))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for n in a[2]:
            assert torch.equal(a[2][n], b[2][n]), n


def test_stream_argument(s4):
    x = inputs(33, 50, 1, 1, 1, 16, 16, BF)
    d = {n: t.cuda() for n, t in x.items()}
    p = s4.DeltaPlan(1, 50, 1, 1, 16, 16, BF)
    ws, o, new = p.workspace(), torch.empty_like(d["v"]), torch.empty_like(d["state"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    s4.delta_fwd(p, d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], o, new, ws, scale=0.7,
                 stream=st)
    st.synchronize()
    z = {n: t.double() for n, t in x.items()}
    ro, rs = reference(z["q"], z["k"], z["v"], z["g"], z["beta"], z["state"], 0.7, [(0, 50)])
    close(o, ro, "o")
    close(new, rs, "state")


def test_no_tokens(s4):
    x = inputs(34, 0, 3, 1, 2, 8, 8, BF)
    _, _, _, _, o, new = forward(s4, x, 3)
    assert torch.equal(new.cpu(), x["state"])
    _, _, g = backward(s4, x, 3)
    assert torch.equal(g["state"].cpu(), x["dstate_out"])


def test_long_sequence_far_state(s4):
    # 40 chunks with weak decay: the carried state keeps fp32 accuracy
    x = inputs(35, 2560, 1, 1, 1, 64, 16, BF)
    x["g"] *= 0.02
    check_forward(s4, x, 1)


def test_validation_env(s4, monkeypatch):
    monkeypatch.setenv("S4DPLR_VALIDATE", "1")
    x = inputs(36, 20, 1, 1, 1, 8, 8, F32)
    x["g"][3, 0] = -math.inf
    forward(s4, x, 1)
    x["g"][4, 0] = 0.5
    with pytest.raises(s4.S4DPLRPreconditionError):
        forward(s4, x, 1)
    x["g"][4, 0] = -0.5
    x["v"][2, 0, 1] = math.nan
    with pytest.raises(s4.S4DPLRPreconditionError):
        forward(s4, x, 1)


def test_refused_tensors(s4):
    x = inputs(37, 20, 2, 1, 2, 8, 8, BF)
    d = {n: t.cuda() for n, t in x.items()}
    p = s4.DeltaPlan(2, 20, 1, 2, 8, 8, BF, training=True)
    o, new, ws = torch.empty_like(d["v"]), torch.empty_like(d["state"]), p.workspace()

    def call(plan=p, **kw):
        a = dict(q=d["q"], k=d["k"], v=d["v"], g=d["g"], beta=d["beta"], state=d["state"], o=o,
                 state_out=new, ws=ws)
        s = {n: kw.pop(n) for n in ("saved", "offsets") if n in kw}
        a.update(kw)
        s4.delta_fwd(plan, *a.values(), **s)

    call()
    for bad in (dict(q=d["q"].float()), dict(g=d["g"].double()), dict(state=d["state"].to(BF)),
                dict(k=None), dict(offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=d["q"][:10]), dict(k=d["k"].cpu()), dict(o=o[:, :1]),
                dict(v=d["v"].transpose(0, 1).contiguous().transpose(0, 1)),
                dict(v=d["v"][:1].expand(20, -1, -1)), dict(beta=d["beta"].t()),
                dict(g=d["g"].t().contiguous().t()), dict(ws=ws[:-256]),
                dict(saved=p.saved()[:-256]),
                dict(offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**bad)
    for status, bad in ((6, dict(o=d["v"])), (6, dict(state_out=d["state"].view(-1).as_strided(
            d["state"].shape, d["state"].stride()))), ):
        if bad.get("state_out") is not None:
            call(**bad)                      # the same memory: in place
            continue
        with pytest.raises(s4.S4DPLRError) as e:
            call(**bad)
        assert e.value.status == status
    plain = s4.DeltaPlan(2, 20, 1, 2, 8, 8, BF)
    with pytest.raises(ValueError):
        plain.saved()
    with pytest.raises(s4.S4DPLRError) as e:
        call(plan=plain, saved=p.saved())
    assert e.value.status == 4
    plain.close()
    with pytest.raises(ValueError):
        call(plan=plain)
    odd = s4.DeltaPlan(3, 20, 1, 2, 8, 8, BF)
    with pytest.raises(s4.S4DPLRError) as e:
        call(plan=odd, state=None, state_out=None, ws=odd.workspace())
    assert e.value.status == 2               # 20 rows are no three equal sequences
