"""The workspace of distillation without a GPU: what rows that are cut into chunks
need, which does not grow with the rows beyond those that are, and does for less."""
import pytest

from test_layer_ops_abi_cpu import E_DEVICE, E_SHAPE, distill, lib, no_gpu  # noqa: F401

MOST_V, MOST_K = 1 << 22, 1024


def test_many_rows_need_no_more(lib):
    f = lib.forge_distill_workspace
    for T, V, K in ((65536, 32000, 1024), (16384, 16384, 256), (1 << 30, 1000, MOST_K), (4096, 128256, 64),
                    (1 << 18, MOST_V, MOST_K)):
        assert 16 <= f(T, V, K) == f(1000, V, K) < 1 << 23


def test_a_larger_workspace_does_for_less(lib):
    f = lib.forge_distill_workspace
    rows, columns, entries = (0, 1, 10, 64, 65, 192, 193, 256, 257, 400, 401, 1000, 1 << 18), (
        0, 1, 100, 4096, 4097, 16384, 16385, 65537, 131073, MOST_V), (0, 1, 5, 512, MOST_K)
    for T in rows:
        for V in columns:
            sizes = [f(T, V, K) for K in entries]
            assert sizes == sorted(sizes)
        for K in entries:
            sizes = [f(T, V, K) for V in columns]
            assert sizes == sorted(sizes)
    for V in columns:
        for K in entries:
            sizes = [f(T, V, K) for T in rows]
            assert sizes == sorted(sizes)


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
        assert distill(lib, ws_bytes=1 << 23, **kw) == E_DEVICE
        assert distill(lib, ws_bytes=lib.forge_distill_workspace(1000, V, 5), **kw) == E_DEVICE
    need = lib.forge_distill_workspace(64, 20000, 5)
    assert distill(lib, T=64, V=20000, ld=20000, ws_bytes=need) == E_DEVICE
    assert distill(lib, T=64, V=20000, ld=20000, ws_bytes=need - 1) == E_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,zt", [(1000, 3000, "float32"), (700, 40000, "bfloat16"), (600, 70001, "float32"),
                                    (500, 140000, "bfloat16")])
def test_rows_of_any_number_with_the_workspace_of_many(T, V, zt):
    import torch

    import weight_gradient_gemm_amd as wg
    from test_gpu_distill import check, inputs
    z, u, ids, weight, V = inputs(torch, T, V, 1024 if V < 5000 else 20, zt)
    n = wg.library().forge_distill_workspace(T, V, u.shape[1])
    ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for t in (T, 260, 100, 20, 1):
        check(torch, wg, (z[:t], u[:t], ids[:t], weight[:t], V), workspace=ws[2048:2048 + n])
        assert bool((ws[:2048] == 0xA5).all() and (ws[2048 + n:] == 0xA5).all())
