"""The workspace of distillation without a GPU: what rows that are cut into chunks
need, and no more than the least one where no row is."""
import pytest

from test_layer_ops_abi_cpu import E_DEVICE, E_SHAPE, distill, lib, no_gpu  # noqa: F401

MOST_V, MOST_K = 1 << 22, 1024


def test_many_rows_need_none(lib):
    f = lib.forge_distill_workspace
    for T, V, K in ((65536, 32000, 1024), (16384, 16384, 256), (1 << 30, 1000, MOST_K), (4096, 128256, 64),
                    (1 << 18, MOST_V, MOST_K)):
        assert f(T, V, K) == 16


def test_few_rows(lib):
    """A chunk's two numbers and an entry's logit in float32; never more than 8 MB."""
    f = lib.forge_distill_workspace
    for T in (1, 8, 64):
        for V in (20000, 70000, 128256):
            assert f(T, V, 100) == T * ((V + 4095) // 4096 * 8 + 400)
    assert max(f(T, MOST_V, MOST_K) for T in range(0, 3000)) < 1 << 23


def test_no_call_is_asked_for_more(lib):
    no_gpu()
    for T, V in ((1000, 100), (300000, 128), (5000, 128256)):
        ld, far = (V + 7) // 8 * 8, 1 << 45
        kw = dict(T=T, V=V, ld=ld, z=far, grad=2 * far, u=3 * far, ids=4 * far, w=5 * far, loss=6 * far, ws=7 * far)
        assert distill(lib, ws_bytes=16, **kw) == E_DEVICE
        assert distill(lib, ws_bytes=15, **kw) == E_SHAPE
    need = lib.forge_distill_workspace(64, 20000, 5)
    assert distill(lib, T=64, V=20000, ld=20000, ws_bytes=need) == E_DEVICE
    assert distill(lib, T=64, V=20000, ld=20000, ws_bytes=need - 1) == E_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,zt", [(1000, 3000, "float32"), (700, 40000, "bfloat16"), (600, 70001, "float32"),
                                    (500, 140000, "bfloat16")])
def test_rows_with_the_least_workspace(T, V, zt):
    import torch

    import weight_gradient_gemm_amd as wg
    from test_gpu_distill import check, inputs
    args = inputs(torch, T, V, 1024 if V < 5000 else 20, zt)
    ws = torch.full((4096,), 0xA5, dtype=torch.uint8, device="cuda")
    assert wg.library().forge_distill_workspace(T, V, 1024) == 16
    check(torch, wg, args, workspace=ws[2048:2064])
    assert bool((ws[:2048] == 0xA5).all() and (ws[2064:] == 0xA5).all())
