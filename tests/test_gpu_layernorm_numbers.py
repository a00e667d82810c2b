"""Layer norm where its numbers are hard."""
import pytest

from test_gpu_layernorm import (HALF, ROW, TINY, U, backward64, check_backward, check_forward,
                                forward64, inputs, within)


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


# --------------------------------------------------------------------------
# the mean's sum in 64 bits
# --------------------------------------------------------------------------
def mean_tolerance(x):
    """Rows' means as they are promised: float64 sums of d values, off by up to d steps of
    2^-53 of the magnitudes, and one rounding."""
    x = x.double()
    return U * x.mean(1).abs() + (x.shape[1] + 2) * 2.0 ** -53 * x.abs().mean(1) + TINY["float32"]


def cancelling_rows(torch, d, dtype, device):
    """Small values with large ones of either sign between them that cancel: neighbours,
    the halves of a row, and a few of them far apart; and a mean far from zero."""
    g = torch.Generator().manual_seed(d)
    x = torch.randn(5, d, generator=g)
    big = 2.0 ** 21 * (1 + torch.rand(5, d // 2, generator=g))
    x[0, 0::2] += big[0]
    x[0, 1::2] -= big[0]
    x[1, : d // 2] += big[1]
    x[1, d // 2:] -= big[1]
    x[2, 0], x[2, d // 2 - 1], x[2, d // 2], x[2, d - 1] = 3e7, 1e7, -1e7, -3e7
    x[3] += 1e4
    x[4, 0::4] += big[4, : (d + 3) // 4]
    x[4, 2::4] -= big[4, : (d + 1) // 4]
    return x.to(getattr(torch, dtype)).to(device)


NUMBERS = [8, 264, 1000, 1024, 2048, 4096, 5000, 8200, 16384, 16392, 40000]


@pytest.mark.gpu
@pytest.mark.parametrize("xt", list(HALF))
@pytest.mark.parametrize("d", NUMBERS)
def test_mean_is_summed_in_64_bits(env, d, xt):
    torch, wg = env
    x = cancelling_rows(torch, d, xt, "cuda")
    gamma, beta = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    y, mean, rstd = torch.empty(5, d, device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    wg.forge_layernorm(x, gamma, beta, y, mean, rstd)
    tol = mean_tolerance(x)
    within(torch, mean, x.double().mean(1), tol, "mean")
    # And y, which a mean that is off shifts as a whole (see forward64 for the other terms).
    want = forward64(torch, x, gamma, beta, 1e-5, "float32")
    r = want[2][:, None]
    n = want[0]
    e_rstd = (ROW / 2 + 6) * U + tol[:, None] ** 2 * r * r / 2
    within(torch, y, n, n.abs() * (e_rstd + 4 * U) + 1.01 * r * tol[:, None] + TINY["float32"], "y")


@pytest.mark.parametrize("d", NUMBERS)
def test_a_float32_sum_is_seen(d):
    """The bound above against sums in float32, and in float64 without its low word, of the
    same rows: both are far outside."""
    import torch
    x = cancelling_rows(torch, d, "float32", "cpu")
    want, tol = x.double().mean(1), mean_tolerance(x)
    lanes = x[:, : d // 8 * 8].view(5, -1, 8)                    # 8 values on end to a thread
    thread = torch.zeros(5, lanes.shape[1])
    for k in range(8):
        thread = thread + lanes[:, :, k]
    float32 = thread.sum(1) / d
    assert int(((float32.double() - want).abs() > tol).sum()) >= 3
    half = (lanes.double().sum(2).view(torch.int64) & ~0xFFFFFFFF).view(torch.float64).sum(1) / d
    assert d == 8 or int(((half - want).abs() > tol).sum()) >= 2


# --------------------------------------------------------------------------
# sums over the rows
# --------------------------------------------------------------------------
def few_rows_tolerance(dY, x, mean, rstd):
    """Rows that each are a workgroup's only one: its dY n is off by the roundings of the
    deviation, of n and of the product, its dY not at all; what adds the rows up rounds once."""
    y = dY.double()
    n = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    size = (y * n).abs().sum(0)
    T = x.shape[0]
    tiny = T * TINY["float32"]
    return (3.01 * U * size + U * (y * n).sum(0).abs() + T * 2.0 ** -52 * size + tiny,
            U * y.sum(0).abs() + T * 2.0 ** -52 * y.abs().sum(0) + TINY["float32"])


@pytest.mark.gpu
@pytest.mark.parametrize("xt,yt", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float32", "bfloat16")])
@pytest.mark.parametrize("T", [1, 2, 9, 63, 64, 65, 100, 128])
@pytest.mark.parametrize("d", [2056, 4096, 8200, 16384])
def test_rows_are_added_up_without_loss(env, T, d, xt, yt):
    """Up to 128 rows of more than 2048 columns: dbeta is the sum rounded once."""
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, T, d, xt, yt, seed=T)
    _, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32")
    _, dg, db = check_backward(torch, wg, dY, x, gamma, mean, rstd)
    want = backward64(torch, dY, x, gamma, mean, rstd, xt)
    e_g, e_b = few_rows_tolerance(dY, x, mean, rstd)
    within(torch, db, want[2], e_b, "dbeta")
    within(torch, dg, want[1], e_g, "dgamma")


# --------------------------------------------------------------------------
# large tensors
# --------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(4500001, 512), (2300003, 1000), (1100001, 2048), (560003, 4096), (280001, 8192),
                                 (140003, 16384), ((1 << 20) + 37, 16392)])
def test_offsets_beyond_32_bits(env, T, d):
    """More than 2^31 elements and 2^32 bytes of each tensor; the last of these has more
    rows than the launches of long rows have workgroups. All rows are zeros but a few, of the
    first, of those around 2^31 elements and 2^32 bytes, and of the last."""
    torch, wg = env
    assert T * d > 1 << 31
    at = [r for c in (0, (1 << 31) // d, (1 << 32) // d, T) for r in range(c - 8, c + 8) if 0 <= r < T]
    at = torch.tensor(sorted(set(at)), device="cuda")
    some, gamma, beta, dY = inputs(torch, len(at), d, "bfloat16", "bfloat16", seed=d)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[at] = some
    y = torch.full_like(x, 7.0)
    mean, rstd = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    wg.forge_layernorm(x, gamma, beta, y, mean, rstd)
    want = forward64(torch, some, gamma, beta, 1e-5, "bfloat16")
    within(torch, y[at], want[0], want[3], "y")
    within(torch, mean[at], want[1], want[4], "mean")
    within(torch, rstd[at], want[2], want[5], "rstd")
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[at] = False
    assert not mean[others].any() and bool((rstd[others] == rstd[others][0]).all())
    zero_row = y[int(torch.nonzero(others)[0])].clone()          # beta, rounded
    assert torch.equal(zero_row, beta.bfloat16())
    y[at] = zero_row
    step = (1 << 28) // d
    assert all(bool((y[r:r + step] == zero_row).all()) for r in range(0, T, step))
    # Backward in place: dY is zero elsewhere, and so are dX and what is added up.
    y.zero_()
    y[at] = dY
    dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    wg.forge_layernorm_backward(y, x, gamma, mean, rstd, y, dg, db)
    want = backward64(torch, dY, some, gamma, mean[at], rstd[at], "bfloat16")
    for got, k, what in ((y[at], 0, "dX"), (dg, 1, "dgamma"), (db, 2, "dbeta")):
        within(torch, got, want[k], want[3 + k], what)
    y[at] = 0
    assert not any(bool(y[r:r + step].any()) for r in range(0, T, step))
