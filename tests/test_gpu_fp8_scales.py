"""GPU tests of the 8-bit product at the ends of its scales, and of few rows by many columns.

Scales of 2^-127 (byte 0), whose float32 is subnormal, and of 2^127 (byte 254) meet in one product,
so that the result is of ordinary size.  A float32 output widens the values first: they are drawn
so that each stands for a normal bf16 number.  Tolerances as in test_gpu_fp8: (K + 16) 2^-24 of the sum
of magnitudes for float32; 2^-12 of it and the rounding of the output for 16 bits."""
import pytest
import torch

from test_gpu_fp8 import check_product, operands

pytestmark = pytest.mark.gpu

BF, F32, F16, F64 = torch.bfloat16, torch.float32, torch.float16, torch.float64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("M,N,K,square", [(5, 20, 256, False), (130, 70, 384, False), (200, 260, 640, True)])
def test_ends_of_the_scales(s4, dtype, M, N, K, square):
    gen = torch.Generator().manual_seed(M + N + K)
    groups = K // 128
    sign = lambda *n: torch.randint(0, 2, n, generator=gen).double() * 2 - 1
    a = (2 + 14 * torch.rand(M, K, generator=gen, dtype=F64)) * sign(M, K)       # 2^-127 a is normal
    b = (0.25 + 1.5 * torch.rand(N, K, generator=gen, dtype=F64)) * sign(N, K)   # 2^127 b is finite
    a, b = a.to(E4M3), b.to(E4M3)
    sa = torch.randint(0, 3, (M, groups), generator=gen).to(torch.uint8)
    tall = -(-N // 128) if square else N
    sb = torch.randint(250, 255, (tall, groups), generator=gen).to(torch.uint8)
    out = torch.empty(M, N, dtype=dtype, device="cuda")
    s4.matmul_fp8(a.cuda(), sa.view(E8M0).cuda(), b.cuda(), sb.view(E8M0).cuda(), out)
    torch.cuda.synchronize()
    wide = lambda s: torch.exp2(s.double() - 127).repeat_interleave(128, 1)
    av = a.double() * wide(sa)
    sbw = wide(sb).repeat_interleave(128, 0)[:N] if square else wide(sb)
    bv = b.double() * sbw
    want, size = av @ bv.T, av.abs() @ bv.abs().T
    if dtype == F32:
        tol = (K + 16) * 2.0 ** -24 * size
    else:
        tol = 2.0 ** -12 * size + torch.finfo(dtype).eps / 2 * want.abs() + torch.finfo(dtype).tiny
        assert size.max() < torch.finfo(dtype).max
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [F32, BF, F16])
@pytest.mark.parametrize("M,N,K", [(1, 4100, 300), (16, 5000, 256), (17, 6001, 1000), (32, 4112, 129), (33, 5000, 640),
                                   (64, 8192, 144), (64, 8200, 256), (40, 9003, 100)])
def test_few_rows_by_many_columns(s4, dtype, M, N, K):
    """Whole numbers without a tolerance, as in test_gpu_fp8, and values of many sizes."""
    check_product(s4, operands(M + N, M, N, K, False, True), dtype, True)
    check_product(s4, operands(M + K, M, N, K, True, True), dtype, True)
    if dtype != F16:   # their results pass fp16's range
        check_product(s4, operands(M, M, N, K, False, False, 8), dtype, False)
