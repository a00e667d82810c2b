"""8-bit products of few rows on both sides of the lengths up to which the kernel that cuts
the contraction takes them, and of operands beyond 2^31 bytes through that kernel."""
import pytest

from test_gpu_fp8_block import TILES, check_product, into, operands, random_operand, some_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


@pytest.mark.parametrize("M", [1, 4, 5, 16, 17, 33, 64, 65])
@pytest.mark.parametrize("N", [4096, 4104, 8192, 8200, 12288, 12296])
def test_lengths_on_both_sides(env, M, N):
    torch, wg = env
    A, B = operands(torch, wg, M, N, 520, M + N, "e4m3", "e5m2")
    for tile in (TILES[0], TILES[1]):
        out, ok = into(torch, M, N)
        wg.forge_matmul_fp8_block(A, B, out, tile=tile)
        check_product(torch, out, A, B)
        assert ok()


@pytest.mark.parametrize("M,N,K", [(3, 12288, 180096), (16, 8184, 270336), (50, 4096, 540672)])
def test_an_operand_beyond_31_bits(env, M, N, K):
    # 2.2 GB of codes: rows of the long operand give what they give in a short one.
    torch, wg = env
    g = torch.Generator(device="cuda").manual_seed(4)
    A, B = random_operand(torch, wg, g, M, K), random_operand(torch, wg, g, N, K)
    assert B.codes.numel() > 1 << 31
    out, ok = into(torch, M, N)
    wg.forge_matmul_fp8_block(A, B, out)
    assert ok()
    for r in (0, (N // 2) // 128 * 128, (N - 1) // 128 * 128):
        part = some_rows(wg, B, r, min(16, N - r))
        check_product(torch, out[:, r:r + part.rows], A, part)
