"""GPU tests of the root-mean-square norm, forward and backward, against 64-bit formulas.

Tolerances.  u = 2^-24.  A lane adds at most 32 squares one after another and then joins 64 lanes and
16 waves (10 additions), so mean h^2 is off by 48 u at most, all terms being positive, and
rstd by half of that and its own square root, quotient and additions: 32 u.  y has two more products
and the rounding to its type, eps / 2.  In dx the row's sum of w xh is off by 56 u of
the sum of magnitudes, each other term by a few u of itself.  dgamma adds each row once:
(rows + 16) u of the sum of magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32, F16, F64 = torch.bfloat16, torch.float32, torch.float16, torch.float64
U = 2.0 ** -24
TINY = {BF: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}   # half the least subnormal


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def inputs(seed, rows, D, dtype):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    return {"x": rnd(rows, D).to(dtype), "residual": (rnd(rows, D) * (1 + 2 * rnd(rows, 1).abs())).to(dtype),
            "gamma": (1 + 0.1 * rnd(D)).float(), "dy": rnd(rows, D).to(dtype), "dh": rnd(rows, D).to(dtype)}


def guarded(n, dtype, off=3):
    """A GPU view of n elements inside a larger buffer of known bytes, at an odd element."""
    size = torch.empty(0, dtype=dtype).element_size()
    store = torch.full(((n + off + 5) * size,), 0x5A, dtype=torch.uint8, device="cuda")
    t = store.view(dtype)[off:off + n]
    return store, t, (off * size, (off + n) * size)


def untouched(store, span):
    return bool((store[:span[0]] == 0x5A).all() and (store[span[1]:] == 0x5A).all())


def reference(x, eps, residual=True, gamma=True):
    h = x["x"].double()
    if residual:
        h = (h + x["residual"].double()).to(x["x"].dtype).double()
    r = (h.square().mean(1, keepdim=True) + eps) ** -0.5
    return h, r, h * r * (x["gamma"].double() if gamma else 1)


def near(got, want, lim, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, worst {float(((got - want).abs() / lim).max()):.2f}"


SIZES = [(1, 1), (3, 7), (1, 128), (5, 129), (2, 255), (4, 512), (7, 1000), (64, 1024), (3, 1025),
         (9, 2048), (5, 4097), (2, 8192), (3, 12000), (2, 16384), (2, 16388), (2, 32768), (2, 32767)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("residual,gamma", [(True, True), (False, False)])
def test_forward(s4, dtype, rows, D, residual, gamma):
    x = inputs(rows * 40000 + D, rows, D, dtype)
    dev = {n: t.cuda() for n, t in x.items()}
    hs, h, hspan = guarded(rows * D, dtype)
    ys, y, yspan = guarded(rows * D, dtype)
    rstd = torch.empty(rows, device="cuda")
    s4.rms_norm_fwd(dev["x"], dev["residual"] if residual else None, dev["gamma"] if gamma else None,
                    h.view(rows, D), y.view(rows, D), rstd, eps=1e-5)
    torch.cuda.synchronize()
    wh, wr, wy = reference(x, 1e-5, residual, gamma)
    assert torch.equal(h.view(rows, D).cpu().double(), wh)
    near(rstd, wr[:, 0], 32 * U * wr[:, 0], "rstd")
    near(y.view(rows, D), wy, (torch.finfo(dtype).eps / 2 + 36 * U) * wy.abs() + TINY[dtype], "y")
    assert untouched(hs, hspan) and untouched(ys, yspan)


def scales_of(y, tall=1):
    """The scale of each group of y (64 bits), as a power of two."""
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % 128, 0, -y.shape[0] % tall))
    big = y.abs().unflatten(1, (-1, 128)).unflatten(0, (-1, tall)).amax((1, 3))
    m, e = torch.frexp(big)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(big > 0, k, -126).clamp(min=-126), big


def rounded8(y, k, tall=1):
    """The e4m3 values of y under the scales 2^k."""
    s = torch.exp2(k.double()).repeat_interleave(128, 1)[:, :y.shape[1]].repeat_interleave(tall, 0)[:y.shape[0]]
    u = y / s
    step = torch.exp2((torch.frexp(u).exponent - 1).clamp(min=-6).double() - 3)
    return torch.round(u / step) * step


@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (2, 128), (5, 300), (33, 1024), (3, 1025), (4, 4096),
                                    (2, 8200), (2, 16384), (2, 20000), (1, 32767)])
def test_8_bits_are_those_of_y(s4, rows, D):
    """A float32 y is the value that is rounded to 8 bits: these are equal to the rounding of y."""
    x = inputs(D, rows, D, F32)
    x["residual"][0] = 0
    x["x"][0] *= 1e-30 if rows > 1 else 1
    dev = {n: t.cuda() for n, t in x.items()}
    y = torch.empty(rows, D, device="cuda")
    groups = -(-D // 128)
    qs, q, qspan = guarded(rows * D, torch.float8_e4m3fn)
    ss, sc, sspan = guarded(rows * groups, torch.float8_e8m0fnu)
    s4.rms_norm_fwd(dev["x"], dev["residual"], dev["gamma"], None, y, q=q.view(rows, D),
                    scales=sc.view(rows, groups))
    torch.cuda.synchronize()
    want = y.double().cpu()
    k, _ = scales_of(want)
    assert torch.equal(sc.view(torch.uint8).view(rows, groups).cpu().int() - 127, k.int())
    assert torch.equal(q.view(rows, D).cpu().double(), rounded8(want, k))
    assert untouched(qs, qspan) and untouched(ss, sspan)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("rows,D", [(5, 300), (16, 1024), (3, 4104), (2, 32768)])
def test_8_bits_of_16_bit_rows(s4, dtype, rows, D):
    """Half a step of e4m3 (2^-4, or half of its least step 2^-9 times the scale) beside y's own error;
    the scale is that of the 64-bit y, but where its largest value is that near to a border."""
    x = inputs(D, rows, D, dtype)
    dev = {n: t.cuda() for n, t in x.items()}
    q = torch.empty(rows, D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(rows, -(-D // 128), dtype=torch.float8_e8m0fnu, device="cuda")
    y = torch.empty_like(dev["x"])
    s4.rms_norm_fwd(dev["x"], dev["residual"], dev["gamma"], None, y, q=q, scales=sc)
    torch.cuda.synchronize()
    wy = reference(x, 1e-5)[2]
    k, big = scales_of(wy)
    low, high = scales_of(wy * (1 - 40 * U))[0], scales_of(wy * (1 + 40 * U))[0]
    got = sc.view(torch.uint8).cpu().int() - 127
    assert bool(((got >= low) & (got <= high)).all())
    s = torch.exp2(got.double()).repeat_interleave(128, 1)[:, :D]
    near(q.cpu().double() * s, wy, 36 * U * wy.abs() + torch.maximum((2.0 ** -4) * wy.abs() * (1 + 36 * U),
                                                                     s * 2.0 ** -10), "q")
    near(y, wy, (torch.finfo(dtype).eps / 2 + 36 * U) * wy.abs() + TINY[dtype], "y")


def test_rows_that_are_not_finite(s4):
    x = inputs(1, 4, 300, F32)
    x["x"][1, 200], x["x"][2, 5] = float("nan"), float("inf")
    x["x"][3] = 0
    dev = {n: t.cuda() for n, t in x.items()}
    y, q = torch.empty(4, 300, device="cuda"), torch.empty(4, 300, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, 3, dtype=torch.float8_e8m0fnu, device="cuda")
    s4.rms_norm_fwd(dev["x"], None, dev["gamma"], None, y, q=q, scales=sc)
    y, q, sc = y.cpu(), q.cpu().float(), sc.view(torch.uint8).cpu()
    assert bool(torch.isfinite(y[0]).all()) and bool(torch.isnan(y[1]).all())
    assert bool((sc[1] == 255).all()) and bool(torch.isnan(q[1]).all())
    # an infinity makes rstd 0, so the others are 0 and it is NaN, and with it its group of 8 bits
    assert bool((y[2, 6:] == 0).all()) and bool(torch.isnan(y[2, 5]))
    assert sc[2].tolist() == [255, 1, 1] and bool(torch.isnan(q[2, :128]).all()) and bool((q[2, 128:] == 0).all())
    assert bool((y[3] == 0).all()) and sc[3].tolist() == [1, 1, 1]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (300, 64), (257, 1000), (64, 1024), (5, 4097), (3, 8192),
                                    (3, 12000), (2, 16388), (9, 32768), (2, 32767)])
@pytest.mark.parametrize("dh,gamma", [(True, True), (False, False)])
def test_backward(s4, dtype, rows, D, dh, gamma):
    x = inputs(rows * 50000 + D, rows, D, dtype)
    h, r, _ = reference(x, 1e-5)
    h16, rstd = h.to(dtype).cuda(), r[:, 0].float().cuda()
    dev = {n: t.cuda() for n, t in x.items()}
    ds, dx, dspan = guarded(rows * D, dtype)
    dgamma = torch.empty(D, device="cuda")
    ws = torch.empty(s4.rms_norm_workspace_bytes(h16) + 256, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:]
    call = lambda a, b: s4.rms_norm_bwd(h16, dev["gamma"] if gamma else None, rstd, dev["dy"],  # noqa: E731
                                        dev["dh"] if dh else None, a, b, ws)
    call(dx.view(rows, D), dgamma)
    torch.cuda.synchronize()
    r = rstd.double().cpu()[:, None]
    xh, dy = h * r, x["dy"].double()
    w = dy * (x["gamma"].double() if gamma else 1)
    norm = r * (w - xh * (w * xh).mean(1, keepdim=True))
    top = x["dh"].double() if dh else torch.zeros_like(dy)
    lim = torch.finfo(dtype).eps / 2 * (top + norm).abs() + TINY[dtype]
    lim = lim + U * (4 * top.abs() + r * (10 * w.abs() + 62 * xh.abs() * (w * xh).abs().mean(1, keepdim=True)))
    near(dx.view(rows, D), top + norm, lim, "dx")
    near(dgamma, (dy * xh).sum(0), (rows + 16) * U * (dy * xh).abs().sum(0), "dgamma")
    assert untouched(ds, dspan)
    # each alone, the same bits; dx in the place of dh
    alone, first = torch.empty_like(dgamma), dx.clone()
    call(None, alone)
    assert torch.equal(alone, dgamma)
    if dh:
        s4.rms_norm_bwd(h16, dev["gamma"] if gamma else None, rstd, dev["dy"], dev["dh"], dev["dh"], None, ws)
        assert torch.equal(dev["dh"].flatten(), first)


def test_gradient_by_differences(s4):
    """The forward pass's own difference quotient: h0 + t d, in float32, with t = 2^-7."""
    x = inputs(4, 3, 40, F32)
    gen = torch.Generator().manual_seed(9)
    d = torch.randn(3, 40, generator=gen, dtype=F64)
    loss = lambda t: float((reference({**x, "x": x["x"].double() + t * d, "residual": x["residual"].double()},  # noqa: E731
                                      1e-5)[2] * x["dy"].double()).sum())
    t = 2.0 ** -12
    want = (loss(t) - loss(-t)) / (2 * t)
    h, r, _ = reference(x, 1e-5)
    dev = {n: v.cuda() for n, v in x.items()}
    h, rstd, dx = h.float().cuda(), torch.empty(3, device="cuda"), torch.empty(3, 40, device="cuda")
    s4.rms_norm_fwd(dev["x"], dev["residual"], dev["gamma"], h, torch.empty_like(h), rstd)
    ws = torch.empty(s4.rms_norm_workspace_bytes(h), dtype=torch.uint8, device="cuda")
    s4.rms_norm_bwd(h, dev["gamma"], rstd, dev["dy"], None, dx, None, ws)
    got = float((dx.double().cpu() * d).sum())
    # third derivatives times t^2 / 6 (t^2 = 6e-8) and float32's own errors
    assert abs(got - want) <= 1e-4 * float((dx.double().cpu() * d).abs().sum())


def test_in_place_and_empty(s4):
    x = inputs(2, 9, 520, BF)
    dev = {n: t.cuda() for n, t in x.items()}
    h, y, y2 = (torch.empty_like(dev["x"]) for _ in range(3))
    s4.rms_norm_fwd(dev["x"], dev["residual"], dev["gamma"], h, y)
    s4.rms_norm_fwd(dev["x"], dev["residual"], dev["gamma"], dev["residual"], y2)
    assert torch.equal(dev["residual"], h) and torch.equal(y, y2)
    s4.rms_norm_fwd(dev["x"].view(3, 3, 520), None, None, None, y.view(3, 3, 520))
    none = torch.empty(0, 520, dtype=BF, device="cuda")
    dgamma = torch.ones(520, device="cuda")
    s4.rms_norm_fwd(none, none, dev["gamma"], none, none)
    ws = torch.empty(s4.rms_norm_workspace_bytes(none), dtype=torch.uint8, device="cuda")
    s4.rms_norm_bwd(none, dev["gamma"], torch.empty(0, device="cuda"), none, None, none, dgamma, ws)
    assert bool((dgamma == 0).all())


def test_graph_and_stream(s4):
    x = inputs(3, 64, 1024, BF)
    dev = {n: t.cuda() for n, t in x.items()}
    h, y, dx = (torch.empty_like(dev["x"]) for _ in range(3))
    rstd, dgamma = torch.empty(64, device="cuda"), torch.empty(1024, device="cuda")
    ws = torch.empty(s4.rms_norm_workspace_bytes(h), dtype=torch.uint8, device="cuda")

    def step():
        s4.rms_norm_fwd(dev["x"], dev["residual"], dev["gamma"], h, y, rstd)
        s4.rms_norm_bwd(h, dev["gamma"], rstd, dev["dy"], dev["dh"], dx, dgamma, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6, 7):
        for n, t in inputs(seed, 64, 1024, BF).items():
            dev[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, y, rstd, dx, dgamma)]
        for t in (h, y, rstd, dx, dgamma):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, y, rstd, dx, dgamma)))


def test_refusals(s4):
    x = torch.ones(4, 256, device="cuda")
    y, q = torch.empty_like(x), torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, 2, dtype=torch.float8_e8m0fnu, device="cuda")
    for bad in (dict(y=None), dict(y=None, q=q), dict(scales=sc), dict(q=q)):
        with pytest.raises(s4.S4DPLRError):
            s4.rms_norm_fwd(x, None, None, None, **{"y": y, **bad})
    for bad in (dict(q=q.float(), scales=sc), dict(q=q, scales=sc.view(torch.uint8)), dict(residual=x.half()),
                dict(h=y.double())):
        with pytest.raises(TypeError):
            s4.rms_norm_fwd(x, bad.pop("residual", None), None, bad.pop("h", None), y, **bad)
    for bad in (dict(q=q, scales=sc[:, :1]), dict(rstd=torch.empty(5, device="cuda")), dict(residual=x[:, :128])):
        with pytest.raises(ValueError):
            s4.rms_norm_fwd(x, bad.pop("residual", None), None, None, y, **bad)
    with pytest.raises(s4.S4DPLRError) as e:
        s4.rms_norm_fwd(x, None, None, y, y)
    assert e.value.status == 6
