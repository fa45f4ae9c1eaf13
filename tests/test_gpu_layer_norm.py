"""GPU tests of the layer norm (layer_norm_fwd, layer_norm_bwd) against its
formula in 64 bits, its reverse-mode gradients and central differences.

Tolerances: an output of b bits is rounded once (eps / 2 of the value).  Before
that: a mean of D values is a tree of at most 32 serial additions a lane and
about 10 across lanes, so off by at most 42 * 2^-24 of the mean magnitude; y, dx
and rstd follow with a few roundings more: 64 * 2^-24 of the largest value in the
row.  dgamma and dbeta are sums over the rows by at most a few hundred serial
additions a lane, whose independent errors add up as the square root of their
number: off by the same part of the sum of magnitudes."""
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


def make(shape, D, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return ((0.5 + 2 * rnd(*shape)).to(dtype), 1 + 0.3 * rnd(D), 0.3 * rnd(D),
            rnd(*shape).to(dtype))


def formula(x, gamma, beta, eps, axis):
    x = x.movedim(axis, -1)
    m = x.mean(-1, keepdim=True)
    r = ((x - m).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (x - m) * r
    return (xh * gamma + beta).movedim(-1, axis), m[..., 0], r[..., 0]


def close(got, ref, name, size=None, factor=1.0):
    """size: the magnitude that the fp32 part of the error goes by."""
    assert got.shape == ref.shape, name
    if ref.numel() == 0:
        return
    got = got.cpu()
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    size = ref.abs().max() if size is None else size
    lim = half * ref.abs() + factor * 64 * UNIT * size + 1e-30
    if got.dtype == F16:
        lim = lim + 2.0 ** -25
    worst = float(((got.double() - ref).abs() / lim).max())
    assert worst <= 1, f"{name}: {worst:.2f} of the tolerance"


def run(s4, x, gamma, beta, dy, axis, eps=1e-5, affine=True, skip=()):
    d = "cuda"
    x, gamma, beta, dy = x.to(d), gamma.to(d), beta.to(d), dy.to(d)
    stat = tuple(n for i, n in enumerate(x.shape) if i != axis % x.dim())
    y = torch.full_like(x, 7.0)
    mean, rstd = torch.full(stat, 7.0, device=d), torch.full(stat, 7.0, device=d)
    gm, bt = (gamma, beta) if affine else (None, None)
    s4.layer_norm_fwd(x, gm, bt, y, mean, rstd, eps=eps, axis=axis)
    ws = torch.empty(s4.layer_norm_workspace_bytes(x, axis), dtype=torch.uint8, device=d)
    g = {"dx": torch.full_like(x, 7.0), "dgamma": torch.full_like(gamma, 7.0),
         "dbeta": torch.full_like(gamma, 7.0)}
    g = {n: None if n in skip else t for n, t in g.items()}
    s4.layer_norm_bwd(x, gm, mean, rstd, dy, g["dx"], g["dgamma"], g["dbeta"], ws, axis=axis)
    return y, mean, rstd, g


def check(s4, shape, axis, dtype, seed=0, eps=1e-5, affine=True, data=None):
    D = shape[axis]
    x, gamma, beta, dy = make(shape, D, dtype, seed)
    if data is not None:
        x = data.to(dtype)
    if not affine:
        gamma, beta = torch.ones(D), torch.zeros(D)
    y, mean, rstd, g = run(s4, x, gamma, beta, dy, axis, eps, affine)
    X = x.double().requires_grad_()
    G, B = gamma.double().requires_grad_(), beta.double().requires_grad_()
    ry, rm, rr = formula(X, G, B, eps, axis)
    big = lambda t: t.detach().abs().amax(axis, keepdim=True)  # noqa: E731
    spread = (big(X) * rr.detach().unsqueeze(axis)).clamp(min=1)
    close(y, ry.detach(), "y", spread * G.detach().abs().max() + B.detach().abs().max())
    close(mean, rm.detach(), "mean", big(X).squeeze(axis))
    close(rstd, rr.detach(), "rstd", rr.detach() * spread.squeeze(axis))
    dx, dg, db = torch.autograd.grad((ry * dy.double()).sum(), [X, G, B])
    size = rr.detach().unsqueeze(axis) * big(dy.double() * 1) * G.detach().abs().max() * spread * spread
    close(g["dx"], dx, "dx", size)
    over = [i for i in range(x.dim()) if i != axis % x.dim()]
    a = dy.double().abs()
    close(g["dgamma"], dg, "dgamma", (a * spread).sum(over))
    close(g["dbeta"], db, "dbeta", a.sum(over))


WIDTHS = [1, 2, 7, 8, 63, 64, 65, 255, 257, 511, 512, 513, 1000, 1024, 1025, 2047, 2049, 4096, 4099,
          8192, 8193, 16384, 16385, 32767, 32768]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF, F16])
def test_rows(s4, D, dtype):
    check(s4, (5, D), -1, dtype, seed=D)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 63, 2047, 2049, 5001])
def test_row_counts(s4, rows):
    check(s4, (rows, 100), -1, F32, seed=rows)
    check(s4, (rows, 2049), -1, BF, seed=rows)


@pytest.mark.parametrize("D", [16392, 32765])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_wide_rows_left_out(s4, D, dtype):
    x, gamma, beta, dy = make((517, D), D, dtype, 3)
    full = run(s4, x, gamma, beta, dy, -1)[3]
    for skip in (("dx",), ("dgamma",), ("dgamma", "dbeta")):
        part = run(s4, x, gamma, beta, dy, -1, skip=skip)[3]
        assert all(part[n] is None or torch.equal(part[n], full[n]) for n in full)
    X, g = x[500:].double(), dy.double()
    r = ((X - X.mean(1, keepdim=True)).square().mean(1, keepdim=True) + 1e-5).rsqrt()
    xh = (X - X.mean(1, keepdim=True)) * r
    w = g[500:] * gamma.double()
    ref = r * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    spread = xh.abs().amax(1, keepdim=True)
    close(full["dx"][500:], ref, "dx", r * w.abs().amax(1, keepdim=True) * spread * spread)
    a = g.abs().sum(0)
    close(full["dbeta"], g.sum(0), "dbeta", a)


def test_wide_rows_of_no_batch(s4):
    x, gamma, beta, dy = make((0, 20000), 20000, BF, 3)
    g = run(s4, x, gamma, beta, dy, -1)[3]
    assert bool((g["dgamma"] == 0).all()) and bool((g["dbeta"] == 0).all())


def test_leading_dimensions(s4):
    check(s4, (3, 5, 2, 96), 3, BF)
    check(s4, (2, 3, 48, 7), 2, F32)
    check(s4, (40, 5), 0, F32)


@pytest.mark.parametrize("D", [1, 2, 8, 63, 64, 65, 256, 257, 511, 513, 600])
@pytest.mark.parametrize("outer,inner", [(3, 65), (1, 1000), (70, 2), (2, 3)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_channels(s4, D, outer, inner, dtype):
    check(s4, (outer, D, inner), 1, dtype, seed=D + inner)


@pytest.mark.parametrize("D", [5, 70, 256, 300, 515])
@pytest.mark.parametrize("dtype,inner", [(BF, 1024), (F16, 1026), (BF, 1023), (F32, 1028)])
def test_channels_of_many_positions(s4, D, dtype, inner):
    check(s4, (33, D, inner), 1, dtype, seed=D)


@pytest.mark.parametrize("D,dtype,affine", [(65, BF, True), (3, F32, False)])
def test_channels_of_more_tiles_than_blocks(s4, D, dtype, affine):
    # 84 copies of a batch that the other tests' sizes cover
    x, gamma, beta, dy = make((100, D, 1000), D, dtype, 5)
    y, mean, rstd, g = run(s4, x, gamma, beta, dy, 1, affine=affine)
    Y, M, R, G = run(s4, x.cuda().repeat(84, 1, 1), gamma, beta, dy.cuda().repeat(84, 1, 1), 1,
                     affine=affine)
    for one, all_ in ((y, Y), (mean, M), (rstd, R), (g["dx"], G["dx"])):
        assert bool((all_.unflatten(0, (84, 100)) == one).all())
    # 8.4e6 terms, 512 of them (131 250 tiles, 256 blocks) after one another a lane: errors
    # of 2^-24 each add up to sqrt(512) < 64 of them
    for n, a in (("dbeta", dy.double().abs().sum((0, 2))),):
        close(G[n], 84 * dy.double().sum((0, 2)), n, 84 * a)


@pytest.mark.parametrize("D", [64, 256, 300])
def test_channels_of_no_batch(s4, D):
    x, gamma, _, _ = make((0, D, 5), D, F32, 1)
    x, gamma = x.cuda(), gamma.cuda()
    st = torch.empty(0, 5, device="cuda")
    dg, db = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
    ws = torch.full((s4.layer_norm_workspace_bytes(x, 1),), 77, dtype=torch.uint8, device="cuda")
    s4.layer_norm_fwd(x, gamma, None, torch.empty_like(x), st, st, axis=1)
    s4.layer_norm_bwd(x, gamma, st, st, x, torch.empty_like(x), dg, db, ws, axis=1)
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_channels_half(s4):
    check(s4, (4, 33, 129), 1, F16)


def test_many_tiles(s4):
    # more tiles of positions, and of rows, than blocks of the backward pass
    check(s4, (40, 24, 1024), 1, F32)
    check(s4, (40, 700, 1024), 1, BF)
    check(s4, (9000, 136), -1, F32)


@pytest.mark.parametrize("shape,axis", [((6, 200), 1), ((6, 3000), 1), ((3, 40, 50), 1)])
def test_large_offset(s4, shape, axis):
    # a common offset of 1000 deviations costs only the offset's own rounding
    gen = torch.Generator().manual_seed(1)
    data = torch.randn(shape, generator=gen) + 1000
    check(s4, shape, axis, F32, data=data)


@pytest.mark.parametrize("shape,axis", [((6, 200), 1), ((3, 40, 50), 1)])
@pytest.mark.parametrize("eps", [1e-5, 0.5])
def test_constant_vectors(s4, shape, axis, eps):
    # variance 0: y = beta, rstd = 1 / sqrt(eps)
    check(s4, shape, axis, F32, data=torch.full(shape, 0.25), eps=eps)


@pytest.mark.parametrize("shape,axis", [((6, 200), 1), ((3, 40, 50), 1)])
def test_without_gain(s4, shape, axis):
    check(s4, shape, axis, BF, affine=False)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape,axis", [((6, 200), 1), ((3, 40, 50), 1)])
def test_bad_value_stays_in_its_vector(s4, value, shape, axis):
    x, gamma, beta, dy = make(shape, shape[1], F32, 3)
    want = run(s4, x, gamma, beta, dy, axis)
    z = x.clone()
    if len(shape) == 2:
        z[2, 5] = value
        hit = (2, slice(None))
    else:
        z[1, 5, 7] = value
        hit = (1, slice(None), 7)
    got = run(s4, z, gamma, beta, dy, axis)
    for a, b in ((got[0], want[0]), (got[3]["dx"], want[3]["dx"])):
        assert bool(a[hit].isnan().all())
        a, b = a.clone(), b.clone()
        a[hit] = b[hit] = 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 65, 1001])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_any_alignment(s4, D, dtype):
    x, gamma, beta, dy = make((9, D), D, dtype, 4)
    want = run(s4, x, gamma, beta, dy, -1)
    pad = lambda t: torch.cat([t.flatten()[:1], t.flatten()]).cuda()[1:].view(t.shape)  # noqa: E731
    got = run(s4, pad(x), pad(gamma), pad(beta), pad(dy), -1)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    for n in got[3]:
        assert torch.equal(got[3][n], want[3][n])


@pytest.mark.parametrize("shape,axis", [((6, 200), 1), ((6, 5000), 1), ((3, 40, 50), 1),
                                        ((3, 700, 50), 1)])
def test_in_place(s4, shape, axis):
    x, gamma, beta, _ = (t.cuda() for t in make(shape, shape[1], BF, 5))
    y = torch.empty_like(x)
    s4.layer_norm_fwd(x, gamma, beta, y, axis=axis)
    s4.layer_norm_fwd(x, gamma, beta, x, axis=axis)
    assert torch.equal(x, y)


@pytest.mark.parametrize("skip", [("dx",), ("dgamma",), ("dbeta",), ("dgamma", "dbeta"),
                                  ("dx", "dgamma", "dbeta")])
@pytest.mark.parametrize("shape", [(50, 300), (50, 3001), (5, 40, 70), (5, 300, 70)])
def test_gradients_left_out(s4, skip, shape):
    x, gamma, beta, dy = make(shape, shape[1], BF, 6)
    full = run(s4, x, gamma, beta, dy, 1)[3]
    some = run(s4, x, gamma, beta, dy, 1, skip=skip)[3]
    for n, t in some.items():
        assert (t is None) == (n in skip)
        assert t is None or torch.equal(t, full[n]), n


def test_gradients_against_differences(s4):
    """Central differences of the 64-bit loss with h = 1e-4: off by about 1e-8 of
    a loss that is smooth at scale 1; the gradient's own error is ``close``'s."""
    for shape, axis in (((7, 90), 1), ((3, 20, 11), 1)):
        x, gamma, beta, dy = make(shape, shape[1], F32, 8)
        g = run(s4, x, gamma, beta, dy, axis)[3]
        gen = torch.Generator().manual_seed(2)
        for i, n in enumerate(("dx", "dgamma", "dbeta")):
            z = [x.double(), gamma.double(), beta.double()]
            e = torch.randn(z[i].shape, generator=gen, dtype=torch.float64)
            loss = []
            for h in (1e-4, -1e-4):
                v = list(z)
                v[i] = z[i] + h * e
                loss.append(float((formula(*v, 1e-5, axis)[0] * dy.double()).sum()))
            mine = g[n].double().cpu() * e
            assert abs(float(mine.sum()) - (loss[0] - loss[1]) / 2e-4) <= 1e-5 * float(
                mine.abs().sum()), n


@pytest.mark.parametrize("shape,axis", [((0, 64), 1), ((0, 8, 5), 1), ((3, 8, 0), 1)])
def test_nothing_to_do(s4, shape, axis):
    x, gamma, beta, dy = make(shape, shape[1], F32, 0)
    y, _, _, g = run(s4, x, gamma, beta, dy, axis)
    assert bool((g["dgamma"] == 0).all()) and bool((g["dbeta"] == 0).all())


@pytest.mark.parametrize("shape", [(64, 1024), (8, 64, 100)])
def test_graph_replays(s4, shape):
    D = shape[1]
    x, gamma, beta, dy = (t.cuda() for t in make(shape, D, BF, 9))
    stat = (shape[0],) + shape[2:]
    y, mean, rstd = torch.empty_like(x), torch.empty(stat).cuda(), torch.empty(stat).cuda()
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    ws = torch.empty(s4.layer_norm_workspace_bytes(x, 1), dtype=torch.uint8, device="cuda")

    def call():
        s4.layer_norm_fwd(x, gamma, beta, y, mean, rstd, axis=1)
        s4.layer_norm_bwd(x, gamma, mean, rstd, dy, dx, dg, db, ws, axis=1)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    outs = [y, mean, rstd, dx, dg, db]
    for i in range(4):
        nx, _, _, ndy = make(shape, D, BF, 20 + i)
        x.copy_(nx)
        dy.copy_(ndy)
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


def test_agrees_with_the_block_norm(s4):
    """The channel layout's norm against the oracle's block pre-norm."""
    import numpy as np
    x, gamma, beta, _ = make((2, 48, 64), 48, F32, 10)
    y = torch.empty_like(x, device="cuda")
    s4.layer_norm_fwd(x.cuda(), gamma.cuda(), beta.cuda(), y, axis=1)
    v = x.double().numpy()
    m, var = v.mean(1, keepdims=True), v.var(1, keepdims=True)
    ref = (v - m) / np.sqrt(var + 1e-5) * gamma.numpy()[:, None] + beta.numpy()[:, None]
    assert float(np.abs(y.cpu().numpy() - ref).max()) <= 64 * UNIT * float(np.abs(ref).max())


def test_refused_tensors(s4):
    x, gamma, beta, dy = (t.cuda() for t in make((6, 32), 32, BF, 0))
    y, st = torch.empty_like(x), torch.empty(6, device="cuda")
    ws = torch.empty(s4.layer_norm_workspace_bytes(x), dtype=torch.uint8, device="cuda")
    for bad in ((x.double(), gamma, beta, y), (x, gamma.to(BF), beta, y), (x, gamma, beta, y.float()),
                (None, gamma, beta, y)):
        with pytest.raises(TypeError):
            s4.layer_norm_fwd(*bad)
    for bad in ((x.t(), gamma[:6], beta[:6], y), (x, gamma[:5], beta, y), (x, gamma, beta, y[:3]),
                (x.cpu(), gamma, beta, y), (x, gamma.cpu(), beta, y)):
        with pytest.raises(ValueError):
            s4.layer_norm_fwd(*bad)
    with pytest.raises(ValueError):
        s4.layer_norm_fwd(x, gamma, beta, y, axis=2)
    with pytest.raises(ValueError):
        s4.layer_norm_fwd(x, gamma, beta, y, mean=st[:5])
    for eps in (-1.0, float("nan")):
        with pytest.raises(s4.S4DPLRError) as e:
            s4.layer_norm_fwd(x, gamma, beta, y, eps=eps)
        assert e.value.status == 2
    with pytest.raises(s4.S4DPLRError) as e:
        s4.layer_norm_fwd(x, gamma, beta, y, mean=st, rstd=st)
    assert e.value.status == 6
    with pytest.raises(ValueError):
        s4.layer_norm_bwd(x, gamma, st, st, dy, y, None, None, ws[:-1])
    with pytest.raises(s4.S4DPLRError) as e:
        s4.layer_norm_bwd(x, gamma, st, st, dy, dy, None, None, ws)
    assert e.value.status == 6
    wide = torch.empty(2, 32769, device="cuda")
    with pytest.raises(s4.S4DPLRError) as e:
        s4.layer_norm_fwd(wide, None, None, torch.empty_like(wide))
    assert e.value.status == 2
