"""GPU tests of the 8-bit product by tiles of 128 and of 256, and of quantization in more than 256 tiles,
where a block writes both forms.  Whole numbers without a tolerance, others with that of test_gpu_fp8."""
import pytest
import torch

from test_gpu_fp8 import BF, F16, F32, check, check_product, matrix, operands, quantized, s4  # noqa: F401

pytestmark = pytest.mark.gpu

# at least 256 tiles of 128; rows that are no multiple of 16 bytes are read piece by piece
TILES_128 = [(2050, 2050, 272), (2050, 2050, 129), (2177, 1920, 1296), (1921, 2178, 1003), (2048, 2048, 64),
             (2048, 2048, 24), (2048, 2176, 7)]
# one round of tiles of 256, which 16-bit outputs take
TILES_256 = [(2950, 4000, 272), (4096, 4096, 128), (3841, 3850, 1040), (8000, 1930, 48)]


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("M,N,K", TILES_128 + TILES_256)
@pytest.mark.parametrize("square", [False, True])
def test_products_of_whole_numbers(s4, dtype, M, N, K, square):  # noqa: F811
    check_product(s4, operands(M + N + K, M, N, K, square, True), dtype, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(2050, 2050, 272), (2050, 2050, 1003), (2950, 4000, 400)])
@pytest.mark.parametrize("spread", [0, 8])
def test_products(s4, dtype, M, N, K, spread):  # noqa: F811
    check_product(s4, operands(M + N + K, M, N, K, spread == 0, False, spread), dtype, False)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("rows,cols", [(2100, 2100), (2177, 2049), (2176, 2056), (40, 33000)])
@pytest.mark.parametrize("square", [False, True])
def test_quantize_both_forms_at_once(s4, dtype, rows, cols, square):  # noqa: F811
    x = matrix(rows * 1000 + cols, rows, cols, dtype)
    q, sc, qt, st = quantized(s4, x.cuda(), square)
    tall = 128 if square else 1
    check(x, q, sc, tall)
    check(x.T.contiguous(), qt, st, tall)
