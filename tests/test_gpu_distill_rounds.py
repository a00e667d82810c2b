"""Distillation around whole rounds of workgroups, where rows go from one to a workgroup to
chunks and back."""
import pytest

from test_gpu_distill import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


@pytest.mark.parametrize("zt,gt,V", [("float32", "bfloat16", 100003), ("float32", "float32", 66001),
                                     ("bfloat16", "bfloat16", 131080), ("bfloat16", "float32", 200001)])
def test_rows_on_both_sides(env, zt, gt, V):
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, 657, V, 11, zt, "bfloat16", "int32", seed=8)
    for T in (64, 96, 97, 160, 161, 208, 209, 256, 257, 368, 369, 432, 433, 512, 513, 576, 577, 656, 657):
        check(torch, wg, (z[:T], u[:T], ids[:T], weight[:T], V), gt, 2.0, 1.0 / T)


@pytest.mark.parametrize("T", [270, 560])
def test_in_place_left_out_and_masked(env, T):
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, T, 100003, 11, masked=False, seed=9)
    weight[[0, 256, T - 1]] = 0
    ids[1] = -1
    u[257] = -float("inf")
    z[0, 7] = float("nan")
    keep = z.gather(1, ids.clamp(min=0))
    z[2, : V // 2] = -float("inf")
    z.scatter_(1, ids.clamp(min=0), keep)
    args = (z, u, ids, weight, V)
    loss, apart = check(torch, wg, args)
    assert not loss[[0, 1, 256, 257, T - 1]].any()
    again, same = check(torch, wg, args, in_place=True)
    assert torch.equal(loss, again) and torch.equal(apart, same)
