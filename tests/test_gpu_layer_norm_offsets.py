"""GPU tests of layer_norm_fwd on vectors whose values are large against their spread:
constant ones at values with no short binary form, and low variances far from zero.

With u = 2^-24 (half a step of fp32): a first mean of at most 80 additions after one another is
off by d <= 80 u |x|.  The second pass finds that as a sum of at most K = 2064 additions (32768
channels over 16 waves), so to K u of itself: far below a step, and the corrected mean is off
by its own rounding, half a step, and by 2^-20 of the deviation, below which no
correction is made.  The variance loses K u of its size and of d^2, rstd half
of that part of (variance + eps).  y = (x - mean) rstd gamma + beta then follows the mean's rounding
times rstd."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U, K, EPS = 2.0 ** -24, 2064, 1e-5


@pytest.fixture(scope="module")
def s4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import structured_state_space_dplr_amd as s4
    return s4


ROWS = [(7, D, 1) for D in (100, 513, 1001, 2048, 2051, 4099, 8192, 8195, 16384, 16387, 32765, 32768)]
CHANNELS = [(2, D, 65) for D in (5, 64, 100, 256, 300, 512, 700, 4096, 32768)]


def norm(s4, x, gamma, beta):
    y = torch.empty_like(x)
    stat = (x.shape[0],) + x.shape[2:]
    mean, rstd = torch.empty(stat, device="cuda"), torch.empty(stat, device="cuda")
    s4.layer_norm_fwd(x, gamma, beta, y, mean, rstd, eps=EPS, axis=1)
    return y, mean, rstd


def shaped(x, shape):
    return x.view(shape[:2]) if shape[2] == 1 else x.view(shape)


@pytest.mark.parametrize("shape", ROWS + CHANNELS)
@pytest.mark.parametrize("value", [10.1, -1000.1, 70000.7])
def test_constant_vectors(s4, shape, value):
    x = shaped(torch.full(shape, value, device="cuda"), shape)
    gen = torch.Generator().manual_seed(1)
    gamma, beta = (torch.randn(shape[1], generator=gen).cuda() for _ in range(2))
    y, mean, rstd = norm(s4, x, gamma, beta)
    assert bool((mean == x.flatten()[0]).all()), "mean"
    assert torch.equal(y, beta.view(1, -1, *[1] * (x.dim() - 2)).expand_as(y)), "y"
    rest = (80 * U * abs(value)) ** 2 * 2 * K * U
    err = float((rstd.double() * EPS ** 0.5 - 1).abs().max())
    assert err <= 8 * U + rest / (2 * EPS), err


@pytest.mark.parametrize("shape", ROWS + CHANNELS)
@pytest.mark.parametrize("dtype,base,spread", [(torch.float32, 1000.1, 1e-2), (torch.float32, -77.3, 1e-3),
                                               (torch.float16, 1000.0, 3.0)])
def test_low_variances(s4, shape, dtype, base, spread):
    gen = torch.Generator().manual_seed(shape[1])
    x = shaped((base + spread * torch.randn(shape, generator=gen)).to(dtype), shape)
    gamma = 1 + 0.3 * torch.randn(shape[1], generator=gen)
    y, mean, rstd = (t.cpu() for t in norm(s4, x.cuda(), gamma.cuda(), None))
    X = x.double()
    m = X.mean(1, keepdim=True)
    var = (X - m).square().mean(1, keepdim=True)
    r = (var + EPS).rsqrt()
    step = torch.exp2(torch.floor(torch.log2(m.abs())) - 23)
    far = (mean.unsqueeze(1).double() - m).abs() / step
    near = 2.0 ** -20 * var.sqrt() / step          # at most so many steps are left
    assert bool((far <= 0.55 + near).all()), f"mean: {float(far.max()):.2f} steps"
    off = K * U * (1 + (80 * U * base) ** 2 / (var + EPS)) + 8 * U
    assert bool(((rstd.unsqueeze(1).double() / r - 1).abs() <= off).all()), "rstd"
    g = gamma.double().view(1, -1, *[1] * (x.dim() - 2))
    want = (X - m) * r * g
    lim = (0.55 + near) * step * r * g.abs() + (off + 8 * U) * want.abs()
    if dtype != torch.float32:
        lim = lim + torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -25
    worst = float(((y.double() - want).abs() / lim).max())
    assert worst <= 1, f"y: {worst:.2f} of the tolerance"


@pytest.mark.parametrize("shape", [(6, 2051, 1), (6, 20000, 1), (2, 300, 65), (2, 700, 65)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_statistics_of_a_bad_value(s4, shape, value):
    # what is not finite is not hidden by the correction, and stays in its vector
    x = shaped(torch.ones(shape, device="cuda"), shape)
    x[1, shape[1] - 1] = value
    y, mean, rstd = norm(s4, x, None, None)
    assert bool(y[1].isnan().all()) and bool(rstd[1].isnan().all())
    assert not bool(mean[1].isfinite().any())
    assert bool(y[0].isfinite().all()) and bool(rstd[0].isfinite().all())


@pytest.mark.parametrize("shape", [(64, 1024, 1), (64, 4096, 1), (16, 16384, 1), (4, 256, 65)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_means_near_zero(s4, shape, dtype):
    """Of values that cancel, the mean follows the rounding of their sum: n values in a tree of t
    <= 42 additions after one another, whose errors of u of the partial sums (at most the sum of
    magnitudes) are independent: sqrt(t) u < 8 u of the mean magnitude over its root, here 8 u."""
    gen = torch.Generator().manual_seed(2)
    x = shaped((0.01 + torch.randn(shape, generator=gen)).to(dtype), shape)
    mean = norm(s4, x.cuda(), None, None)[1].cpu().double()
    assert float((mean - x.double().mean(1)).abs().max()) <= 8 * U * float(x.double().abs().mean())
