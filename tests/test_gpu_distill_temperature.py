"""Distillation at temperatures far below 1: the loss is scale tau sum q (du - dz) and
tau^2 times the logarithms of the sums, and tau^2 alone leaves float32's range."""
import pytest

from test_gpu_distill import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


def shifted(torch, T, V):
    """Rows whose largest logit is not the teacher's, so that the loss is of tau's size."""
    z, u, ids, weight, V = inputs(torch, T, V, 6, masked=False)
    z[:, :V] = z[:, :V].roll(1, 1)
    return z, u, ids, weight, V


@pytest.mark.parametrize("tau", [1e-12, 1e-18, 1e-20, 3e-23, 1e-27])
@pytest.mark.parametrize("T,V", [(5, 1000), (300, 9000), (6, 40000), (9, 70000)])
def test_small_temperatures(env, T, V, tau):
    torch, wg = env
    loss, grad = check(torch, wg, shifted(torch, T, V), tau=tau)
    assert (loss > 0.1 * tau).all() and torch.isfinite(loss).all() and torch.isfinite(grad).all()


@pytest.mark.parametrize("tau,scale", [(1e-19, 1e-12), (1e-27, 1e20), (1e20, 1e-30), (3e37, 1e-38), (1e12, 1e-24)])
@pytest.mark.parametrize("T,V", [(5, 1000), (300, 9000), (6, 40000), (9, 70000)])
def test_temperatures_and_scales_far_apart(env, T, V, tau, scale):
    torch, wg = env
    check(torch, wg, shifted(torch, T, V), tau=tau, scale=scale)
