"""GPU tests of quantization to 8 bits and of the 8-bit matrix product.

Quantization is exact but for its one rounding, so it is compared without a tolerance.  Products of
small whole numbers have exact sums in any order and any width, so they are compared without
one too.  Products of arbitrary values: a float32 output adds K exact products in float32, off by
(K + 16) 2^-24 of the sum of their magnitudes at most; a 16-bit output comes from an
instruction that keeps about 13 bits of a group's sum of magnitudes (measured 1.2e-4 < 2^-13
for a single group), so 2^-12 of the sum of magnitudes, and its own rounding eps / 2."""
import pytest
import torch

from test_gpu_rms_norm import guarded, near, rounded8, scales_of, untouched

pytestmark = pytest.mark.gpu

BF, F32, F16, F64 = torch.bfloat16, torch.float32, torch.float16, torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


def groups(n):
    return -(-n // 128)


def quantized(s4, x, square=False, turned=True, plain=True):
    """The four outputs of quantize_fp8 in guarded buffers, on the host."""
    rows, cols = x.shape
    made = []
    for r, c in ((rows, cols), (cols, rows)):
        made += [guarded(r * c, E4M3), guarded((groups(r) if square else r) * groups(c), E8M0)]
    v = [made[0][1].view(rows, cols), made[1][1].view(-1, groups(cols)),
         made[2][1].view(cols, rows), made[3][1].view(-1, groups(rows))]
    s4.quantize_fp8(x, *(v[:2] if plain else (None, None)), *(v[2:] if turned else (None, None)))
    torch.cuda.synchronize()
    for i, (store, t, span) in enumerate(made):
        assert untouched(store, span if (plain if i < 2 else turned) else (0, 0))
    return [t.cpu() for t in v]


def matrix(seed, rows, cols, dtype):
    """Values of many sizes, with zeros, and groups of nothing but zeros."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, dtype=F64) * torch.exp2(
        torch.randint(-12, 13, (rows, cols), generator=gen).double())
    x = x * torch.exp2(torch.randint(-8, 9, (rows, 1), generator=gen).double()) / 2.0 ** (12 if dtype == F16 else 0)
    x[torch.rand(rows, cols, generator=gen) < 0.1] = 0
    if rows > 3:
        x[2] = 0
    return x.to(dtype)


def check(x, q, sc, tall=1):
    x = x.double()
    k, _ = scales_of(x, tall)
    assert torch.equal(sc.view(torch.uint8).int() - 127, k.int())
    assert torch.equal(q.double(), rounded8(x, k, tall))


SIZES = [(1, 1), (1, 128), (128, 1), (3, 7), (127, 129), (128, 128), (130, 257), (300, 40), (33, 1000), (512, 264)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("square", [False, True])
def test_quantize(s4, dtype, rows, cols, square):
    x = matrix(rows * 1000 + cols, rows, cols, dtype)
    q, sc, qt, st = quantized(s4, x.cuda(), square)
    tall = 128 if square else 1
    check(x, q, sc, tall)
    check(x.T.contiguous(), qt, st, tall)


def test_quantize_of_a_column_range(s4):
    wide = matrix(3, 140, 600, BF).cuda()
    for lo, hi in ((1, 301), (64, 192), (599, 600)):
        x = wide[:, lo:hi]
        for plain, turned in ((True, False), (False, True)):
            q, sc, qt, st = quantized(s4, x, plain=plain, turned=turned)
            if plain:
                check(x.cpu(), q, sc)
            else:
                check(x.cpu().T.contiguous(), qt, st)


def test_quantize_at_borders(s4):
    """Largest values on either side of 448 2^k, subnormal numbers, the largest number, ties."""
    x = torch.zeros(12, 128)
    x[0, 0], x[1, 0] = 448 * 2.0 ** 5, 448 * 2.0 ** 5 * (1 + 2.0 ** -23)
    x[2, 0], x[3, 0], x[4, 0] = 2.0 ** -149, 2.0 ** -126, torch.finfo(F32).max
    x[5, 0], x[6, 0], x[7, 0] = -448.0, 2.0 ** -118 * 1.75, 2.0 ** -118 * 1.7500001
    x[8, :9] = torch.tensor([256.0, 8.5, 9.5, 17.0, 19.0, -8.5, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11])
    x[9, 1:3] = torch.tensor([-0.0, 448.0])
    x[10, :2] = torch.tensor([1.0, 2.0 ** -149])
    q, sc, qt, st = quantized(s4, x.cuda())
    check(x, q, sc)
    assert int(sc.view(torch.uint8)[2, 0]) == 1 and int(sc.view(torch.uint8)[11, 0]) == 1
    check(x.T.contiguous(), qt, st)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_quantize_not_finite(s4, what):
    x = torch.ones(130, 300)
    x[1, 200] = what
    q, sc, qt, st = quantized(s4, x.cuda())
    sc, st = sc.view(torch.uint8).int(), st.view(torch.uint8).int()
    assert int(sc[1, 1]) == 255 and int((sc == 255).sum()) == 1
    assert int(st[200, 0]) == 255 and int((st == 255).sum()) == 1
    assert bool(torch.isnan(q[1, 128:256].float()).all()) and int(torch.isnan(q.float()).sum()) == 128
    assert bool(torch.isnan(qt[200, :128].float()).all()) and int(torch.isnan(qt.float()).sum()) == 128


def operands(seed, M, N, K, square, whole, spread=0):
    """8-bit matrices and scales; ``whole``: numbers from -3 to 3 under scales 1/2 to 2."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen)  # noqa: E731
    nb = groups(N) if square else N
    if whole:
        a, b = rnd(-3, 4, M, K).float(), rnd(-3, 4, N, K).float()
        sa, sb = rnd(126, 129, M, groups(K)), rnd(126, 129, nb, groups(K))
    else:
        a, b = (torch.randn(n, K, generator=gen) * 32 * torch.exp2(-rnd(0, spread + 1, n, K).float()) for n in (M, N))
        sa, sb = rnd(107, 140, M, groups(K)), rnd(107, 140, nb, groups(K))
    return [a.to(E4M3).cuda(), sa.to(torch.uint8).view(E8M0).cuda(), b.to(E4M3).cuda(),
            sb.to(torch.uint8).view(E8M0).cuda()]


def values(q, sc):
    s = torch.exp2(sc.view(torch.uint8).double() - 127).repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * s.repeat_interleave(1 if sc.shape[0] == q.shape[0] else 128, 0)[:q.shape[0]]


def check_product(s4, ops, dtype, exact):
    a, sa, b, sb = ops
    (M, K), N = a.shape, b.shape[0]
    store, out, span = guarded(M * N, dtype)
    s4.matmul_fp8(a, sa, b, sb, out.view(M, N))
    torch.cuda.synchronize()
    A, B = values(a, sa).cpu(), values(b, sb).cpu()
    want, mag = A @ B.T, A.abs() @ B.abs().T
    if exact:
        assert torch.equal(out.view(M, N).cpu(), want.to(dtype))
    else:
        lim = (K + 16) * U * mag if dtype == F32 else 2.0 ** -12 * mag + torch.finfo(dtype).eps / 2 * want.abs()
        near(out.view(M, N), want, lim + 2.0 ** -133, "out")
    assert untouched(store, span)


PRODUCTS = [(1, 1, 1), (1, 7, 16), (3, 130, 128), (16, 64, 256), (17, 200, 1000), (32, 512, 2048), (33, 100, 144),
            (64, 384, 640), (65, 33, 130), (100, 520, 1040), (128, 128, 128), (129, 257, 384), (256, 256, 512),
            (300, 1000, 99), (513, 260, 1296), (40, 9, 4104)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("square", [False, True])
def test_products_of_whole_numbers(s4, dtype, M, N, K, square):
    """Sums of at most 4104 products of 9 times 4 are below 2^24 (float32: exact); rounded once."""
    check_product(s4, operands(M + N + K, M, N, K, square, True), dtype, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("spread", [0, 8])
def test_products(s4, dtype, M, N, K, spread):
    check_product(s4, operands(M + N + K, M, N, K, False, False, spread), dtype, False)
    check_product(s4, operands(M + N + K + 1, M, N, K, True, False, spread), dtype, False)


@pytest.mark.parametrize("M,N,K", [(1000, 1500, 512), (2100, 700, 272), (700, 4100, 129)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_tiles(s4, dtype, M, N, K):
    check_product(s4, operands(M, M, N, K, True, True), dtype, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [5, 70, 300])
def test_column_ranges(s4, dtype, M):
    """Operands and result inside wider matrices, at odd places too."""
    for off, K, N in ((16, 256, 130), (3, 200, 130), (0, 144, 64)):
        a, sa, b, sb = operands(M + off, M, N, K, True, True)
        want = values(a, sa).cpu() @ values(b, sb).cpu().T
        wa, wb = (torch.full((n, K + 48), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for n in (M, N))
        wa.view(torch.uint8)[:, off:off + K] = a.view(torch.uint8)
        wb.view(torch.uint8)[:, off:off + K] = b.view(torch.uint8)
        out = torch.full((M, N + 9), 7.0, dtype=dtype, device="cuda")
        s4.matmul_fp8(wa[:, off:off + K], sa, wb[:, off:off + K], sb, out[:, 5:5 + N])
        assert torch.equal(out[:, 5:5 + N].cpu(), want.to(dtype))
        assert bool((out[:, :5] == 7).all()) and bool((out[:, 5 + N:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_values(s4, dtype):
    """NaN scales and values reach their row or column alone; scales at both ends; zeros."""
    for M in (8, 200):
        a, sa, b, sb = operands(7, M, 300, 300, False, True)
        sa.view(torch.uint8)[3, 1] = 255
        b.view(torch.uint8)[17, 40] = 0x7F
        out = torch.empty(M, 300, dtype=dtype, device="cuda")
        s4.matmul_fp8(a, sa, b, sb, out)
        bad = torch.isnan(out).cpu()
        want = torch.zeros_like(bad)
        want[3], want[:, 17] = True, True
        assert torch.equal(bad, want)
        a, sa, b, sb = operands(8, M, 300, 256, False, True)
        sa.view(torch.uint8)[:] = 1
        sb.view(torch.uint8)[:] = 240
        s4.matmul_fp8(a, sa, b, sb, out)
        assert torch.equal(out.cpu(), (values(a, sa).cpu() @ values(b, sb).cpu().T).to(dtype))


def test_empty(s4):
    e = lambda *s: torch.empty(*s, dtype=E4M3, device="cuda")  # noqa: E731
    z = lambda *s: torch.empty(*s, dtype=E8M0, device="cuda")  # noqa: E731
    out = torch.ones(5, 9, device="cuda")
    s4.matmul_fp8(e(5, 0), z(5, 0), e(9, 0), z(9, 0), out)
    assert bool((out == 0).all())
    s4.matmul_fp8(e(0, 64), z(0, 1), e(9, 64), z(9, 1), out[:0])
    s4.quantize_fp8(out[:0], e(0, 9), z(0, 1), e(9, 0), z(9, 0))
    s4.quantize_fp8(out, None, None)


def test_graph(s4):
    """Quantization and the three products of a layer's training step, captured and replayed."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w, dy = (torch.randn(*s, generator=gen, device="cuda").to(BF) for s in ((200, 264), (136, 264), (200, 136)))
    mk = lambda r, c, sq=False: (torch.empty(r, c, dtype=E4M3, device="cuda"),  # noqa: E731
                                 torch.empty(groups(r) if sq else r, groups(c), dtype=E8M0, device="cuda"))
    qx, qxt, qw, qwt = mk(200, 264), mk(264, 200), mk(136, 264, True), mk(264, 136, True)
    qy, qyt = mk(200, 136), mk(136, 200)
    out, dx, dw = torch.empty(200, 136, dtype=BF, device="cuda"), torch.empty_like(x), torch.empty(136, 264, device="cuda")

    def step():
        s4.quantize_fp8(x, *qx, *qxt)
        s4.quantize_fp8(w, *qw, *qwt)
        s4.matmul_fp8(*qx, *qw, out)
        s4.quantize_fp8(dy, *qy, *qyt)
        s4.matmul_fp8(*qy, *qwt, dx)
        s4.matmul_fp8(*qyt, *qxt, dw)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (x, w, dy):
            t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, dx, dw)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (out, dx, dw)))
        X, W, Y = (t.double() for t in (x, w, dy))
        # a value of 8 bits is within 2^-4 of itself: products of two within 2^-3 + 2^-8
        for got, want, mag in ((out, X @ W.T, X.abs() @ W.abs().T), (dx, Y @ W, Y.abs() @ W.abs()),
                               (dw, Y.T @ X, Y.T.abs() @ X.abs())):
            assert bool(((got.double() - want).abs() <= (2.0 ** -3 + 2.0 ** -7) * mag + 2.0 ** -8).all())


def test_refusals(s4):
    a, sa, b, sb = operands(1, 8, 200, 256, True, True)
    out = torch.empty(8, 200, device="cuda")
    for bad in ((a.float(), sa, b, sb, out), (a, sa.view(torch.uint8), b, sb, out), (a, sa, b, sb, out.double()),
                (a, sa, b.view(torch.uint8), sb, out), (None, sa, b, sb, out), (a, sa, b, None, out)):
        with pytest.raises(TypeError):
            s4.matmul_fp8(*bad)
    for bad in ((a[:, :128], sa, b, sb, out), (a, sa[:4], b, sb, out), (a, sa, b, sb[:1], out),
                (a, sa, b, sb, out[:, :100]), (a.T, sa, b, sb, out), (a.cpu(), sa, b, sb, out)):
        with pytest.raises(ValueError):
            s4.matmul_fp8(*bad)
    x = torch.ones(200, 300, device="cuda")
    q, sc = torch.empty(200, 300, dtype=E4M3, device="cuda"), torch.empty(200, 3, dtype=E8M0, device="cuda")
    qt, sq = torch.empty(300, 200, dtype=E4M3, device="cuda"), torch.empty(3, 2, dtype=E8M0, device="cuda")
    with pytest.raises(ValueError, match="both"):
        s4.quantize_fp8(x, q, sc, qt, sq)
    with pytest.raises(TypeError):
        s4.quantize_fp8(x.double(), q, sc)
    with pytest.raises(TypeError):
        s4.quantize_fp8(x, q, None)
    with pytest.raises(ValueError):
        s4.quantize_fp8(x, q, sc[:, :2])
    with pytest.raises(ValueError):
        s4.quantize_fp8(x.T, qt, sq)
