"""Layer norm where its numbers are hard."""
import pytest

from test_gpu_layernorm import HALF, check_backward, check_forward, inputs


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


# --------------------------------------------------------------------------
# squares outside float32's range
# --------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("xt", list(HALF))
@pytest.mark.parametrize("d", [8, 264, 1000, 2048, 4096, 8200, 16392, 24576])
def test_deviations_of_any_size(env, d, xt):
    """Rows of deviations from 1e-36 to 1e35, without an eps and with one as small as their
    squares: the variance is a float64 sum where float32 would lose it."""
    torch, wg = env
    powers = (-118, -100, -70, -63, -52, -50, -48, -20, 0, 40, 62, 64, 66, 100, 116)
    x, gamma, beta, dY = inputs(torch, len(powers), d, "float32", "float32")
    x *= torch.tensor([2.0 ** k for k in powers], device="cuda")[:, None]
    x = x.to(getattr(torch, xt))
    for eps in (0.0, 2.0 ** -126, 2.0 ** -100, 1e-5):
        y, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32", eps=eps)
        assert torch.isfinite(y).all() and (rstd > 0).all()
        if eps == 0.0:
            check_backward(torch, wg, dY, x, gamma, mean, rstd)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [8, 1000, 4096, 24576])
def test_equal_values_without_eps(env, d):
    """A variance of zero is no small variance: NaN, as in the formula, and its row's alone."""
    torch, wg = env
    x, gamma, beta, _ = inputs(torch, 7, d)
    x[2], x[4] = 5.0, 0.0
    x[3] *= 2.0 ** -90
    y, rstd = torch.empty_like(x), torch.empty(7, device="cuda")
    wg.forge_layernorm(x, gamma, beta, y, None, rstd, eps=0.0)
    assert torch.isnan(y[[2, 4]]).all() and torch.isfinite(y[[0, 1, 3, 5, 6]]).all()
    assert torch.isinf(rstd[[2, 4]]).all()
