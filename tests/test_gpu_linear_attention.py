"""GPU tests of linear attention with decay (linear_attention_fwd, linear_attention_bwd) against
the recurrence token by token in 64 bits, its reverse, and central differences.

Tolerances: an output of b bits is rounded once (half a step: eps / 2 of the value).  Before
that, every value is a chain of fp32 sums of at most dk + 2 * 64 terms per chunk, whose
rounding errors (2^-24 of the largest term each, independent of each other) add up as the square
root of their number: at most sqrt(384) < 20 per sum, three sums after one another per chunk,
and what a chunk adds to the state fades like the state itself.  64 * 2^-24 of the largest
value of the output allows for that.  dg is a running sum, in 64 bits, of q . dq and k . dk of
at most 512 tokens behind a segment's edge: errors of a few 2^-24 (8) of the sums of
magnitudes, sqrt(2 * 512) = 32 of them: 256 * 2^-24 of the largest such sum."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24
BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def inputs(seed, tokens, S, Hk, Hv, dk, dv, dtype, state=True, gates="token"):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda t: t / (t.norm(dim=-1, keepdim=True) + 1e-6)  # noqa: E731
    x = {"q": unit(rnd(tokens, Hk, dk)), "k": unit(rnd(tokens, Hk, dk)), "v": rnd(tokens, Hv, dv)}
    x = {n: t.to(dtype) for n, t in x.items()}
    x["g"] = (-torch.nn.functional.softplus(rnd(tokens, Hv) - 2)).float()
    if gates == "head":
        x["g"] = -torch.exp(2 * rnd(Hv) - 3).float()
    if gates is None:
        x["g"] = None
        x["v"] = (x["v"].double() / max(tokens, 1) ** 0.5).to(dtype)
    x["state"] = 0.3 * rnd(S, Hv, dk, dv).float() if state else None
    x["dout"] = rnd(tokens, Hv, dv).to(dtype)
    x["dstate_out"] = 0.3 * rnd(S, Hv, dk, dv).float()
    return x


def bounds_of(S, tokens, offsets):
    if offsets is None:
        n = tokens // S
        return [(i * n, i * n + n) for i in range(S)]
    return list(zip(offsets[:-1], offsets[1:]))


def reference(x, S, offsets=None, scale=0.7, gradients=False):
    """Outputs in 64 bits; with gradients also those, and the sums of magnitudes behind dg."""
    z = {n: None if t is None else t.double() for n, t in x.items()}
    tokens, Hk, dk = z["q"].shape
    Hv, dv = z["v"].shape[1:]
    heads = torch.arange(Hv) // (Hv // Hk)
    q, k, v = z["q"][:, heads], z["k"][:, heads], z["v"]
    a = torch.ones(tokens, Hv, dtype=torch.float64) if z["g"] is None else z["g"].exp().expand(tokens, Hv)
    state = torch.zeros(S, Hv, dk, dv, dtype=torch.float64) if z["state"] is None else z["state"]
    o, last = torch.zeros(tokens, Hv, dv, dtype=torch.float64), state.clone()
    r = {n: torch.zeros(tokens, Hv, d, dtype=torch.float64) for n, d in (("dq", dk), ("dk", dk), ("dv", dv))}
    dg, ds = torch.zeros(tokens, Hv, dtype=torch.float64), z["dstate_out"].clone()
    for s, (lo, hi) in enumerate(bounds_of(S, tokens, offsets)):
        line = [state[s]]
        for t in range(lo, hi):
            line.append(line[-1] * a[t][:, None, None] + k[t][:, :, None] * v[t][:, None, :])
            o[t] = scale * (line[-1] * q[t][:, :, None]).sum(1)
        last[s] = line[-1]
        if not gradients:
            continue
        Z = ds[s]
        for t in range(hi - 1, lo - 1, -1):
            r["dq"][t] = scale * (line[t - lo + 1] * z["dout"][t][:, None, :]).sum(2)
            Z = Z + scale * q[t][:, :, None] * z["dout"][t][:, None, :]
            r["dk"][t] = (Z * v[t][:, None, :]).sum(2)
            r["dv"][t] = (Z * k[t][:, :, None]).sum(1)
            dg[t] = a[t] * (Z * line[t - lo]).sum((1, 2))
            Z = Z * a[t][:, None, None]
        ds[s] = Z
    r.update(o=o, state=last)
    if gradients:
        r["sums"] = max([float((q * r["dq"]).abs().sum(2).max()), float((k * r["dk"]).abs().sum(2).max())]
                        if tokens else [0.0])
        for n in ("dq", "dk"):
            r[n] = r[n].unflatten(1, (Hk, Hv // Hk)).sum(2)
        r["dg"] = None if z["g"] is None else dg.sum(0) if z["g"].dim() == 1 else dg
        r["dstate"] = ds
    return r


def close(got, ref, name, extra=0.0):
    assert got.shape == ref.shape, name
    if ref.numel() == 0:
        return
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    err = (got.double().cpu() - ref).abs()
    lim = half * ref.abs() + 64 * UNIT * max(float(ref.abs().max()), 1e-30) + extra
    if got.dtype == F16:
        lim = lim + 2.0 ** -25          # half a step of its smallest numbers
    worst = float((err / lim).max())
    assert worst <= 1, f"{name}: {worst:.2f} of the tolerance"


def forward(s4, x, S, offsets=None, training=False, scale=0.7, in_place=False, plan=None):
    tokens, Hk, dk = x["q"].shape
    Hv, dv = x["v"].shape[1:]
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    p = plan or s4.LinearAttentionPlan(S, tokens, Hk, Hv, dk, dv, x["v"].dtype, training=training)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o = torch.full((tokens, Hv, dv), 7.0, dtype=x["v"].dtype, device="cuda")
    new = d["state"] if in_place else torch.full((S, Hv, dk, dv), 7.0, device="cuda")
    saved = p.saved() if training else None
    s4.linear_attention_fwd(p, d["q"], d["k"], d["v"], d["g"], d["state"], o, new, p.workspace(),
                            saved=saved, scale=scale, offsets=off)
    return p, d, off, saved, o, new


def inside_of(S, tokens, offsets):
    inside = torch.zeros(tokens, dtype=torch.bool)
    for a, b in bounds_of(S, tokens, offsets):
        inside[a:b] = True
    return inside


def check_forward(s4, x, S, offsets=None, **kw):
    tokens = x["q"].shape[0]
    o, new = forward(s4, x, S, offsets, **kw)[4:]
    ref, inside = reference(x, S, offsets), inside_of(S, tokens, offsets)
    close(o[inside.cuda()], ref["o"][inside], "o")
    close(new, ref["state"], "state")
    assert bool((o[~inside.cuda()] == 7.0).all()), "rows outside every sequence were written"


def backward(s4, x, S, offsets=None, scale=0.7, dstate=True, fwd=None, drop=()):
    p, d, off, saved, o, new = fwd or forward(s4, x, S, offsets, training=True, scale=scale)
    out = {n: torch.full(d[n].shape, 7.0, dtype=d[n].dtype, device="cuda") for n in ("q", "k", "v")}
    out = {"d" + n: t for n, t in out.items()}
    out["dg"] = None if d["g"] is None else torch.full_like(d["g"], 7.0)
    out["dstate"] = torch.full_like(new, 7.0)
    out = {n: None if n in drop else t for n, t in out.items()}
    s4.linear_attention_bwd(p, d["q"], d["k"], d["v"], d["g"], saved, d["dout"],
                            d["dstate_out"] if dstate else None, out["dq"], out["dk"], out["dv"],
                            out["dg"], out["dstate"], p.workspace(), scale=scale, offsets=off)
    return out


def check_backward(s4, x, S, offsets=None, dstate=True):
    tokens = x["q"].shape[0]
    got = backward(s4, x, S, offsets, dstate=dstate)
    if not dstate:
        x = dict(x, dstate_out=torch.zeros_like(x["dstate_out"]))
    ref, inside = reference(x, S, offsets, gradients=True), inside_of(S, tokens, offsets)
    at = inside.cuda()
    for n in ("dq", "dk", "dv"):
        close(got[n][at], ref[n][inside], n)
        assert bool((got[n][~at] == 7.0).all()), n
    close(got["dstate"], ref["dstate"], "dstate")
    if x["g"] is None:
        return
    per = x["g"].dim() == 2
    extra = 256 * UNIT * ref["sums"] * (1 if per else tokens ** 0.5)
    close(got["dg"][at] if per else got["dg"], ref["dg"][inside] if per else ref["dg"], "dg", extra)
    if per:
        assert bool((got["dg"][~at] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 63, 64, 65, 150, 256, 257, 700])
def test_lengths(s4, dtype, T):
    check_forward(s4, inputs(T, 2 * T, 2, 2, 2, 32, 16, dtype), 2)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (40, 72), (64, 17), (65, 16), (64, 128), (128, 128),
                                   (128, 200), (129, 33), (250, 70), (256, 256)])
@pytest.mark.parametrize("T", [3, 70, 300])
def test_head_sizes(s4, dtype, dk, dv, T):
    check_forward(s4, inputs(dk * 7 + dv, T, 1, 1, 2, dk, dv, dtype), 1)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 5), (3, 3), (2, 6)])
@pytest.mark.parametrize("T", [5, 100])
def test_head_groups(s4, Hk, Hv, T):
    check_forward(s4, inputs(Hv, 3 * T, 3, Hk, Hv, 24, 40, BF), 3)


OFFSETS = [[0, 0, 1, 65, 65, 200], [3, 20, 20, 130, 131, 190], [0, 200, 200, 200, 200, 200],
           [0, 0, 0, 0, 0, 0], [0, 16, 33, 34, 97, 161], [0, 300, 300, 301, 900, 1000], [5, 600, 610, 618, 1200, 1456],
           [1, 258, 516, 774, 1032, 1289], [0, 256, 512, 768, 1024, 1280]]


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gates", ["token", "head", None])
def test_packed(s4, offsets, dtype, gates):
    x = inputs(offsets[-1], offsets[-1] + 5, 5, 1, 2, 24, 40, dtype, gates=gates)
    check_forward(s4, x, 5, offsets)


@pytest.mark.parametrize("T", [4, 8, 100, 600])
def test_state_in_place_and_none(s4, T):
    check_forward(s4, inputs(T, 2 * T, 2, 1, 2, 48, 32, BF, state=False), 2)
    check_forward(s4, inputs(T, 2 * T, 2, 1, 2, 48, 32, BF), 2, in_place=True)
    check_forward(s4, inputs(T, 2 * T, 2, 1, 2, 48, 32, F32), 2, [0, T + 1, 2 * T], in_place=True)


@pytest.mark.parametrize("dtype", [BF, F32, F16])
@pytest.mark.parametrize("T,dk,dv", [(1, 16, 16), (9, 40, 24), (64, 64, 64), (70, 40, 72), (300, 32, 24),
                                     (130, 128, 128), (70, 200, 72), (70, 72, 256), (700, 16, 40)])
def test_gradients(s4, dtype, T, dk, dv):
    check_backward(s4, inputs(T + dk, T, 1, 2, 2, dk, dv, dtype), 1)


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("gates", ["token", "head", None])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradients_packed(s4, offsets, gates, dtype):
    x = inputs(offsets[-1] + 1, offsets[-1] + 5, 5, 1, 3, 24, 40, dtype, gates=gates)
    check_backward(s4, x, 5, offsets)


@pytest.mark.parametrize("T", [40, 600])
def test_gradients_without_states(s4, T):
    check_backward(s4, inputs(T, 2 * T, 2, 2, 2, 32, 32, BF, state=False), 2, dstate=False)


@pytest.mark.parametrize("T", [40, 600])
def test_each_gradient_alone(s4, T):
    """Outputs that are left out change no bit of the others, and dstate may lie over dstate_out."""
    x = inputs(T, 2 * T, 2, 1, 2, 32, 40, F32)
    fwd = forward(s4, x, 2, training=True)
    names = ("dq", "dk", "dv", "dg", "dstate")
    every = backward(s4, x, 2, fwd=fwd)
    for n in names:
        only = backward(s4, x, 2, fwd=fwd, drop=[m for m in names if m != n])
        assert torch.equal(only[n], every[n]), n
    p, d, off, saved = fwd[:4]
    ds, out = d["dstate_out"].clone(), {n: torch.empty_like(every[n]) for n in names[:4]}
    s4.linear_attention_bwd(p, d["q"], d["k"], d["v"], d["g"], saved, d["dout"], ds, *out.values(), ds,
                            p.workspace(), scale=0.7)
    assert torch.equal(ds, every["dstate"]) and all(torch.equal(out[n], every[n]) for n in out)


@pytest.mark.parametrize("T", [30, 400])
def test_resets(s4, T):
    """g = -infinity and decays far below what fp32 holds: nothing before them is seen, nor has a
    gradient; beside them the gradients keep their digits."""
    x = inputs(T, 2 * T, 2, 1, 2, 24, 24, F32)
    g = x["g"]
    g[T // 2, 0], g[T // 3, 1], g[0, 0], g[T - 1, 0] = -math.inf, -150.0, -math.inf, -1e30
    g[T + 5], g[T + 6] = -math.inf, -math.inf
    check_forward(s4, x, 2)
    check_backward(s4, x, 2)
    dg = backward(s4, x, 2)["dg"].cpu()
    assert bool((dg[torch.isinf(g)] == 0).all())
    assert float(dg[T // 3, 1]) == 0 and float(dg[T - 1, 0]) == 0


def test_differences(s4):
    """Central differences of the forward pass's own float32 outputs in 64-bit formulas."""
    T = 70
    x = inputs(3, T, 1, 1, 2, 8, 8, F32)
    got = backward(s4, x, 1, scale=0.7)
    gen = torch.Generator().manual_seed(1)

    def loss(y):
        r = reference(y, 1)
        return float((r["o"] * x["dout"].double()).sum() + (r["state"] * x["dstate_out"].double()).sum())

    for n, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("state", "dstate")):
        d = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        e = 2.0 ** -13
        up, down = (loss({m: (t.double() + s * e * d if m == n else t) for m, t in x.items()}) for s in (1, -1))
        want = (up - down) / (2 * e)
        have = got[grad].double().cpu() * d
        # e^2 = 1.5e-8 times third derivatives (of g, at most some hundred times the first), and fp32
        assert abs(float(have.sum()) - want) <= 1e-5 * float(have.abs().sum()), n


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("S,T,Hk,Hv,dk,dv", [(1, 5, 2, 2, 64, 48), (2, 200, 2, 2, 64, 48), (1, 300, 1, 3, 128, 64),
                                             (2, 700, 2, 4, 128, 128)])
@pytest.mark.parametrize("training", [False, True])
def test_16_bit_tensors_give_the_fp32_outputs(s4, dtype, S, T, Hk, Hv, dk, dv, training):
    """A value of 16 bits is one of 32, and everything behind the loads is defined in 32 bits."""
    x = inputs(T + dk, S * T, S, Hk, Hv, dk, dv, dtype)
    wide = {n: None if t is None else t.float() for n, t in x.items()}
    a, b = (forward(s4, y, S, training=training) for y in (x, wide))
    assert torch.equal(a[5], b[5]), "state"
    assert torch.equal(a[4], b[4].to(dtype)), "o"
    if training:
        a, b = backward(s4, x, S, fwd=a), backward(s4, wide, S, fwd=b)
        assert torch.equal(a["dstate"], b["dstate"])
        for n in ("dq", "dk", "dv"):
            assert torch.equal(a[n], b[n].to(dtype)), n


def test_prompt_then_tokens(s4):
    """A prompt in two calls and tokens one by one give the whole sequence's outputs."""
    T = 400
    x = inputs(9, T, 1, 1, 2, 40, 24, F32)
    ref = reference(x, 1)
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    state, rows = d["state"].clone(), []
    for lo, hi in [(0, 333), (333, 390)] + [(t, t + 1) for t in range(390, T)]:
        p = s4.LinearAttentionPlan(1, hi - lo, 1, 2, 40, 24, F32)
        o = torch.empty(hi - lo, 2, 24, device="cuda")
        s4.linear_attention_fwd(p, d["q"][lo:hi], d["k"][lo:hi], d["v"][lo:hi], d["g"][lo:hi], state, o, state,
                                p.workspace(), scale=0.7)
        rows.append(o)
    close(torch.cat(rows), ref["o"], "o")
    close(state, ref["state"], "state")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [3, 300])
def test_column_ranges(s4, dtype, T):
    """q, k, v as column ranges of one matrix at odd places."""
    x = inputs(T, T, 1, 2, 2, 24, 40, dtype)
    wide = torch.full((T, 1 + 48 + 48 + 80 + 2), 7.0, dtype=dtype)
    cut = {"q": (1, 49, 24), "k": (49, 97, 24), "v": (97, 177, 40)}
    for n, (a, b, d) in cut.items():
        wide[:, a:b] = x[n].flatten(1)
    wide = wide.cuda()
    whole = forward(s4, x, 1, training=True)
    p, d = whole[:2]
    part = dict(d, **{n: wide[:, a:b].unflatten(1, (2, e)) for n, (a, b, e) in cut.items()})
    o, new, saved = torch.empty_like(whole[4]), torch.empty_like(whole[5]), p.saved()
    s4.linear_attention_fwd(p, part["q"], part["k"], part["v"], part["g"], part["state"], o, new, p.workspace(),
                            saved=saved, scale=0.7)
    assert torch.equal(o, whole[4]) and torch.equal(new, whole[5])
    want = backward(s4, x, 1, fwd=whole)
    got = backward(s4, x, 1, fwd=(p, part, None, saved, o, new))
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_graph(s4):
    """A captured training step against the eager one, with its own eager work in between."""
    T, S = 600, 2
    x = inputs(5, S * T, S, 1, 2, 32, 64, BF)
    p, d, off, saved, o, new = forward(s4, x, S, training=True)
    ws = p.workspace()
    grads = {n: torch.empty_like(d[n]) for n in ("q", "k", "v", "g")}
    ds = torch.empty_like(new)

    def step():
        s4.linear_attention_fwd(p, d["q"], d["k"], d["v"], d["g"], d["state"], o, new, ws, saved=saved)
        s4.linear_attention_bwd(p, d["q"], d["k"], d["v"], d["g"], saved, d["dout"], d["dstate_out"],
                                *grads.values(), ds, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (6, 7, 8):
        for n, t in inputs(seed, S * T, S, 1, 2, 32, 64, BF).items():
            d[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in (o, new, ds, *grads.values())]
        for t in (o, new, ds, *grads.values()):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, (o, new, ds, *grads.values())))


def test_streams(s4):
    """Two calls at once on streams of their own, each with its own workspace."""
    xs = [inputs(i, 1200, 2, 1, 2, 64, 64, BF) for i in (1, 2)]
    want = [forward(s4, x, 2)[4].clone() for x in xs]
    plans = [s4.LinearAttentionPlan(2, 1200, 1, 2, 64, 64, BF) for _ in xs]
    ds = [{n: None if t is None else t.cuda() for n, t in x.items()} for x in xs]
    outs = [torch.empty_like(w) for w in want]
    for p in plans:
        p.workspace()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for p, d, o, s in zip(plans, ds, outs, streams):
            s4.linear_attention_fwd(p, d["q"], d["k"], d["v"], d["g"], d["state"], o, None, p.workspace(),
                                    scale=0.7, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def packed(lengths, first=0):
    return [first] + (torch.tensor(lengths).cumsum(0) + first).tolist()


SHORT = [[9] * 12 + [0] * 20 + [1] * 12, [9, 0] * 40, [0] * 30 + [600] + [0] * 30 + [9, 8, 10] + [1] * 20,
         [8] * 5 + [9] * 5 + [0] * 10, [64, 0, 0, 0, 0, 0, 0, 0, 265] + [0] * 20 + [9],
         [0] * 300 + [7] * 100, [1] * 150 + [700] + [0] * 60, [257] * 6 + [0] * 3 + [256] * 2]


@pytest.mark.parametrize("i", range(len(SHORT)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_short_and_long(s4, i, dtype):
    lengths = SHORT[i]
    offsets = packed(lengths, i % 3)
    check_forward(s4, inputs(i, offsets[-1] + i % 2, len(lengths), 1, 2, 16, 16, dtype), len(lengths), offsets)


@pytest.mark.parametrize("i", [0, 2, 4, 7])
def test_gradients_of_packed_short_and_long(s4, i):
    lengths = SHORT[i]
    offsets = packed(lengths, 1)
    check_backward(s4, inputs(i, offsets[-1], len(lengths), 1, 2, 16, 16, F32), len(lengths), offsets)


@pytest.mark.parametrize("offsets", [[0, 900, 300, 200], [-5, 100, 2000, 900], [900, 0, 0, 900], [2 ** 31 - 1, -2 ** 31, 0, 900],
                                     [0, 899, 1, 900]])
def test_bad_offsets_stay_inside(s4, offsets):
    """Unspecified results, but no access outside the buffers: the guards around them stay."""
    x = inputs(1, 900, 3, 1, 2, 16, 24, BF)
    d = {n: t.cuda() for n, t in x.items()}
    p = s4.LinearAttentionPlan(3, 900, 1, 2, 16, 24, BF, training=True)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def guarded(n, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        store = torch.full((n * size + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
        store = store[-store.data_ptr() % 256:]
        return store, store[256:256 + n * size].view(dtype)

    sizes = {"o": (900 * 2 * 24, BF), "new": (3 * 2 * 16 * 24, F32), "ws": (p.workspace_bytes, torch.uint8),
             "saved": (p.saved_bytes, torch.uint8), "dq": (900 * 16, BF), "dk": (900 * 16, BF),
             "dv": (900 * 2 * 24, BF), "dg": (900 * 2, F32), "ds": (3 * 2 * 16 * 24, F32)}
    b = {n: guarded(*s) for n, s in sizes.items()}
    v = {n: t[1] for n, t in b.items()}
    s4.linear_attention_fwd(p, d["q"], d["k"], d["v"], d["g"], d["state"], v["o"].view(900, 2, 24),
                            v["new"].view(3, 2, 16, 24), v["ws"], saved=v["saved"], offsets=off)
    s4.linear_attention_bwd(p, d["q"], d["k"], d["v"], d["g"], v["saved"], d["dout"], d["dstate_out"],
                            v["dq"].view(900, 1, 16), v["dk"].view(900, 1, 16), v["dv"].view(900, 2, 24),
                            v["dg"].view(900, 2), v["ds"].view(3, 2, 16, 24), v["ws"], offsets=off)
    torch.cuda.synchronize()
    for n, (store, t) in b.items():
        end = 256 + t.numel() * t.element_size()
        assert bool((store[:256] == 0x5A).all()) and bool((store[end:] == 0x5A).all()), n


def test_refusals(s4):
    x = inputs(1, 20, 2, 1, 2, 16, 24, BF)
    p, d, off, saved, o, new = forward(s4, x, 2, training=True)
    call = lambda **kw: s4.linear_attention_fwd(*({**dict(p=p, q=d["q"], k=d["k"], v=d["v"], g=d["g"],  # noqa: E731
                                                          state=d["state"], o=o, new=new, ws=p.workspace()),
                                                   **kw}).values())
    for kw in (dict(p=None), dict(q=d["q"].float()), dict(g=d["g"].half()), dict(v=None), dict(ws=None)):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=d["q"][:10]), dict(g=d["g"][:, :1]), dict(g=d["g"][0, :1]), dict(state=d["state"][:1]),
               dict(o=o.transpose(1, 2)), dict(ws=p.workspace()[:1]), dict(q=d["q"].cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(s4.S4DPLRError) as e:
        call(o=d["v"])
    assert e.value.status == 6
    plain = s4.LinearAttentionPlan(2, 20, 1, 2, 16, 24, BF)
    with pytest.raises(ValueError):
        plain.saved()
    odd = s4.LinearAttentionPlan(3, 20, 1, 2, 16, 24, BF)
    with pytest.raises(s4.S4DPLRError):
        s4.linear_attention_fwd(odd, d["q"], d["k"], d["v"], d["g"], None, o, None, odd.workspace())
    with pytest.raises(s4.S4DPLRError):      # dg where there is no g
        s4.linear_attention_bwd(p, d["q"], d["k"], d["v"], None, saved, d["dout"], None, None, None, None,
                                torch.empty(20, 2, device="cuda"), None, p.workspace())
    with pytest.raises(TypeError):
        s4.LinearAttentionPlan(1, 8, 1, 1, 8, 8, torch.float64)
    closed = s4.LinearAttentionPlan(2, 20, 1, 2, 16, 24, BF)
    ws = closed.workspace()
    closed.close()
    with pytest.raises(ValueError, match="closed"):
        call(p=closed, ws=ws)
