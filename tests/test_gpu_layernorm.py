"""Layer norm and its backward pass on the GPU against the formulas in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                  # half a float32 step, relative
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134}      # half the least step of each type
TYPES = [(x, y) for x in HALF for y in HALF]
# Terms that one float32 sum over a row adds up one after the other: at most 64
# elements of a thread, 6 steps within a wave, 16 waves, and the division.
ROW = 90


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


def inputs(torch, T, d, xt="float32", yt="float32", seed=0, shift=0.3):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = (normal(T, d) * torch.exp(0.7 * normal(d)) + shift * normal(d)).to(getattr(torch, xt))
    dY = (normal(T, d) * 1e-2).to(getattr(torch, yt))
    return x, normal(d) * 0.1 + 1, normal(d) * 0.1, dY


def forward64(torch, x, gamma, beta, eps, out):
    """y, mean, rstd and how far float32 may be off each."""
    x, g = x.double(), gamma.double()
    b = torch.zeros_like(g) if beta is None else beta.double()
    mean = x.mean(1, keepdim=True)
    v = x - mean
    var = (v * v).mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    n = v * rstd
    y = n * g + b
    # A mean that is off by e adds e^2 to the variance: the deviations sum to zero.
    e_mean = ROW * U * x.abs().mean(1, keepdim=True) + U * mean.abs()
    e_rstd = rstd * ((ROW / 2 + 6) * U + e_mean ** 2 / (2 * (var + eps)))
    e_n = v.abs() * e_rstd + rstd * e_mean + 3 * U * n.abs() + e_mean * e_rstd
    e_y = g.abs() * e_n + U * (y.abs() + 2 * b.abs())
    return (y, mean[:, 0], rstd[:, 0],
            e_y * (1 + HALF[out]) + HALF[out] * y.abs() + TINY[out], e_mean[:, 0], e_rstd[:, 0])


def backward64(torch, dY, x, gamma, mean, rstd, out):
    """dX, dgamma, dbeta and how far float32 may be off each."""
    T = x.shape[0]
    y, g = dY.double(), gamma.double()
    r = rstd.double()[:, None]
    n = (x.double() - mean.double()[:, None]) * r
    a = y * g
    c1, c2 = a.mean(1, keepdim=True), (a * n).mean(1, keepdim=True)
    dx = r * (a - c1 - n * c2)
    e1 = (ROW + 2) * U * a.abs().mean(1, keepdim=True)
    e2 = (ROW + 5) * U * (a * n).abs().mean(1, keepdim=True)
    e = r * (e1 + n.abs() * e2 + 6 * U * (a.abs() + c1.abs() + (n * c2).abs()))
    # Rows one after the other: a part's, then 16 groups' shares of 512 parts.
    depth = T / 512 + 72
    return (dx, (y * n).sum(0), y.sum(0), e * (1 + HALF[out]) + HALF[out] * dx.abs() + TINY[out],
            (depth + 4) * U * (y * n).abs().sum(0) + TINY["float32"],
            depth * U * y.abs().sum(0) + TINY["float32"])


def within(torch, got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(),
                           got[bad][:3].tolist(), want[bad][:3].tolist(), tol[bad][:3].tolist())


def guarded(torch, shape, dtype, fill=7.0):
    """A tensor inside a larger one, and a check that nothing around it was written."""
    n = 1
    for k in shape:
        n *= k
    big = torch.full((n + 128,), fill, dtype=getattr(torch, dtype), device="cuda")
    return big[64:64 + n].view(shape), lambda: bool((big[:64] == fill).all() and
                                                    (big[64 + n:] == fill).all())


def check_forward(torch, wg, x, gamma, beta, yt, eps=1e-5, stats=True):
    T, d = x.shape
    y, ok_y = guarded(torch, (T, d), yt)
    mean, ok_m = guarded(torch, (T,), "float32")
    rstd, ok_r = guarded(torch, (T,), "float32")
    wg.forge_layernorm(x, gamma, beta, y, mean if stats else None, rstd if stats else None, eps=eps)
    want = forward64(torch, x, gamma, beta, eps, yt)
    within(torch, y, want[0], want[3], "y")
    if stats:
        within(torch, mean, want[1], want[4], "mean")
        within(torch, rstd, want[2], want[5], "rstd")
    assert ok_y() and ok_m() and ok_r()
    return y, mean, rstd


def check_backward(torch, wg, dY, x, gamma, mean, rstd, bias=True, **kw):
    T, d = x.shape
    xt = str(x.dtype)[6:]
    dX, ok_x = guarded(torch, (T, d), xt)
    dg, ok_g = guarded(torch, (d,), "float32")
    db, ok_b = guarded(torch, (d,), "float32")
    wg.forge_layernorm_backward(dY, x, gamma, mean, rstd, dX, dg, db if bias else None, **kw)
    want = backward64(torch, dY, x, gamma, mean, rstd, xt)
    within(torch, dX, want[0], want[3], "dX")
    within(torch, dg, want[1], want[4], "dgamma")
    if bias:
        within(torch, db, want[2], want[5], "dbeta")
    assert ok_x() and ok_g() and ok_b()
    return dX, dg, db


SIZES = [(1, 8), (1, 4096), (2, 64), (3, 72), (5, 512), (4, 520), (33, 1000), (7, 1024), (9, 1032),
         (6, 2048), (13, 2056), (5, 4096), (3, 4104), (2, 8192), (3, 8200), (2, 16384), (3, 16392),
         (1, 32776), (2, 65536), (333, 1000), (2500, 136), (1500, 2056)]


@pytest.mark.parametrize("T,d", SIZES)
def test_sizes(env, T, d):
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, T, d)
    _, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32")
    check_backward(torch, wg, dY, x, gamma, mean, rstd)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("T,d", [(1, 8), (5, 264), (67, 768), (33, 2008), (18, 4096), (21, 5000),
                                 (9, 12296), (4, 20000), (700, 1144)])
def test_types(env, T, d, xt, yt):
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, T, d, xt, yt, seed=T)
    _, mean, rstd = check_forward(torch, wg, x, gamma, beta, yt)
    check_backward(torch, wg, dY, x, gamma, mean, rstd)


@pytest.mark.parametrize("T,d", [(70001, 8), (9000, 1024), (40000, 256), (5000, 4096), (3000, 8192),
                                 (1100, 16384), (600, 24576), (4099, 1560), (1023, 2048), (511, 4096),
                                 (513, 4104), (4097, 2056), (16387, 520)])
def test_many_rows(env, T, d):
    # Workgroups that go round their loops, parts with unequal numbers of rows.
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, T, d, "bfloat16", "bfloat16", seed=3)
    _, mean, rstd = check_forward(torch, wg, x, gamma, beta, "bfloat16")
    check_backward(torch, wg, dY, x, gamma, mean, rstd)


def test_more_rows_than_workgroups(env):
    # Beyond 2^20 workgroups of four rows each the forward pass loops.
    torch, wg = env
    T, d = (1 << 22) + 3000, 8
    x, gamma, beta, _ = inputs(torch, T, d, "bfloat16")
    check_forward(torch, wg, x, gamma, beta, "bfloat16")


@pytest.mark.parametrize("d", [8, 1000, 4096, 20000])
def test_without_bias_and_statistics(env, d):
    torch, wg = env
    x, gamma, _, dY = inputs(torch, 5, d)
    y, mean, rstd = check_forward(torch, wg, x, gamma, None, "float32")
    y2, _, _ = check_forward(torch, wg, x, gamma, None, "float32", stats=False)
    assert torch.equal(y, y2)
    dX, dg, _ = check_backward(torch, wg, dY, x, gamma, mean, rstd)
    dX2, dg2, db2 = check_backward(torch, wg, dY, x, gamma, mean, rstd, bias=False)
    assert torch.equal(dX, dX2) and torch.equal(dg, dg2) and bool((db2 == 7.0).all())


@pytest.mark.parametrize("d", [8, 264, 4096, 16400])
def test_rows_that_are_hard(env, d):
    """A mean far from zero, rows of equal values, tiny and huge ones."""
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, 6, d)
    x[0] += 1e4
    x[1] = 3.0
    x[2] = 0.0
    x[3] *= 1e-20
    x[4] *= 1e15
    y, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32")
    assert torch.equal(y[1], beta) and torch.equal(y[2], beta)
    assert float(mean[1]) == 3.0
    check_backward(torch, wg, dY, x, gamma, mean, rstd)


@pytest.mark.parametrize("d", [8, 1000, 4096, 8200, 16400])
def test_a_row_that_is_not_finite_stays_alone(env, d):
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, 9, d)
    y, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32")
    dX, _, _ = check_backward(torch, wg, dY, x, gamma, mean, rstd)
    bad = x.clone()
    bad[2, d // 2] = float("nan")
    bad[5, 0] = float("inf")
    y2, m2, r2 = (torch.empty_like(t) for t in (y, mean, rstd))
    wg.forge_layernorm(bad, gamma, beta, y2, m2, r2)
    dX2, dg2, db2 = torch.empty_like(dX), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    wg.forge_layernorm_backward(dY, bad, gamma, m2, r2, dX2, dg2, db2)
    for k in range(9):
        if k in (2, 5):
            assert torch.isnan(y2[k]).any() and torch.isnan(dX2[k]).all()
        else:
            assert torch.equal(y2[k], y[k]) and torch.equal(dX2[k], dX[k])
    assert torch.isnan(dg2).any() and torch.isfinite(db2).all()


def test_eps(env):
    torch, wg = env
    x, gamma, beta, _ = inputs(torch, 4, 136)
    for eps in (0.0, 1e-12, 0.5, 1e6):
        check_forward(torch, wg, x, gamma, beta, "float32", eps=eps)
    x[1] = 2.0
    y = torch.empty_like(x)
    wg.forge_layernorm(x, gamma, beta, y, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2, 3]]).all()


@pytest.mark.parametrize("t", list(HALF))
@pytest.mark.parametrize("T,d", [(7, 1000), (5, 4096), (9, 8192), (3, 24576)])
def test_gradient_in_place(env, T, d, t):
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, T, d, t, t)
    _, mean, rstd = check_forward(torch, wg, x, gamma, beta, t)
    dX, dg, db = check_backward(torch, wg, dY, x, gamma, mean, rstd)
    dg2, db2 = torch.empty_like(dg), torch.empty_like(db)
    wg.forge_layernorm_backward(dY, x, gamma, mean, rstd, dY, dg2, db2)
    assert torch.equal(dY, dX) and torch.equal(dg, dg2) and torch.equal(db, db2)


def test_no_rows(env):
    torch, wg = env
    d = 72
    x = torch.empty(0, d, device="cuda")
    stat = torch.empty(0, device="cuda")
    gamma, dg, db = torch.ones(d, device="cuda"), torch.full((d,), 5.0, device="cuda"), torch.full(
        (d,), 5.0, device="cuda")
    wg.forge_layernorm(x, gamma, None, x, stat, stat)
    wg.forge_layernorm_backward(x, x, gamma, stat, stat, x, dg, db)
    assert (dg == 0).all() and (db == 0).all()


def test_shapes_and_offsets(env):
    """Rows in several dimensions, a vector, and statistics inside a larger array."""
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, 24, 136)
    y, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32")
    y2, stat = torch.empty(2, 3, 4, 136, device="cuda"), torch.zeros(51, device="cuda")
    m2, r2 = stat[1:25].view(2, 3, 4), stat[26:50].view(2, 3, 4)
    wg.forge_layernorm(x.view(2, 3, 4, 136), gamma, beta, y2, m2, r2)
    assert torch.equal(y2.view(24, 136), y) and torch.equal(m2.reshape(-1), mean)
    assert torch.equal(r2.reshape(-1), rstd) and float(stat[[0, 25, 50]].abs().sum()) == 0
    dX, dg, db = check_backward(torch, wg, dY, x, gamma, mean, rstd)
    dX2, dg2 = torch.empty_like(y2), torch.empty_like(dg)
    wg.forge_layernorm_backward(dY.view_as(y2), x.view_as(y2), gamma, m2, r2, dX2, dg2)
    assert torch.equal(dX2.view(24, 136), dX) and torch.equal(dg2, dg)
    one = torch.empty(136, device="cuda")
    wg.forge_layernorm(x[3], gamma, beta, one)
    assert torch.equal(one, y[3])


@pytest.mark.parametrize("T,d", [(600, 264), (37, 4096), (1030, 1032)])
def test_differences(env, T, d):
    """dX, dgamma and dbeta against differences of the forward pass along a direction."""
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, T, d, seed=9)
    _, mean, rstd = check_forward(torch, wg, x, gamma, beta, "float32")
    dX, dg, db = check_backward(torch, wg, dY, x, gamma, mean, rstd)
    g = torch.Generator(device="cuda").manual_seed(5)
    h = 2.0 ** -6
    for which in range(3):
        args = [x, gamma, beta]
        grad = (dX, dg, db)[which]
        step = torch.randn(args[which].shape, generator=g, device="cuda")
        sides, exact, noise = [], [], 0.0
        for sign in (1, -1):
            moved = list(args)
            moved[which] = args[which] + sign * h * step
            y = torch.empty_like(x)
            wg.forge_layernorm(*moved, y)
            want = forward64(torch, *moved, 1e-5, "float32")
            sides.append(float((y.double() * dY.double()).sum()))
            exact.append(float((want[0] * dY.double()).sum()))
            noise += float((want[3] * dY.double().abs()).sum())
            # the step that was taken differs from h by the rounding of the sum
            noise += float((U * moved[which].double().abs() * grad.double().abs()).sum()) * 2
        slope = (sides[0] - sides[1]) / (2 * h)
        slope64 = (exact[0] - exact[1]) / (2 * h)
        tol = noise / (2 * h)
        assert abs(slope - slope64) <= tol
        # What a difference of this width is off the slope by: its third derivative
        # counts h^2 / 6, 256 times less at a sixteenth of the width.
        w = h / 16
        y64 = [forward64(torch, *[a.double() + (s * w * step.double() if k == which else 0)
                                  for k, a in enumerate(args)], 1e-5, "float32")[0] for s in (1, -1)]
        bend = abs(float(((y64[0] - y64[1]) * dY.double()).sum()) / (2 * w) - slope64) * 1.01
        along = float((grad.double() * step.double()).sum())
        tol_grad = backward64(torch, dY, x, gamma, mean, rstd, "float32")[3 + which]
        # The gradients take the stored mean and rstd, off by less than a y is (times
        # gamma, of 0.6 and more): a few sums of e_y |dY| beside the 1 / h = 64 in tol.
        assert abs(slope - along) <= tol + bend + float((tol_grad * step.abs()).sum())


def test_the_same_bits_again(env):
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, 3000, 1544, "bfloat16", "bfloat16")
    first = check_forward(torch, wg, x, gamma, beta, "bfloat16")
    grads = check_backward(torch, wg, dY, x, gamma, *first[1:])
    for _ in range(3):
        again = check_forward(torch, wg, x, gamma, beta, "bfloat16")
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        ws = torch.randint(0, 255, (wg.library().forge_layernorm_workspace(3000, 1544),),
                           device="cuda", dtype=torch.uint8)
        assert all(torch.equal(a, b) for a, b in zip(
            grads, check_backward(torch, wg, dY, x, gamma, *first[1:], workspace=ws)))


def test_captured_and_two_streams(env):
    torch, wg = env
    sets = []
    for seed in (1, 2):
        x, gamma, beta, dY = inputs(torch, 900, 1160, "float32", "bfloat16", seed=seed)
        out = dict(y=torch.empty_like(dY), mean=torch.empty(900, device="cuda"),
                   rstd=torch.empty(900, device="cuda"), dX=torch.empty_like(x),
                   dg=torch.empty(1160, device="cuda"), db=torch.empty(1160, device="cuda"))
        ws = torch.empty(wg.library().forge_layernorm_workspace(900, 1160), dtype=torch.uint8,
                         device="cuda")

        def run(stream=None, x=x, gamma=gamma, beta=beta, dY=dY, o=out, ws=ws):
            wg.forge_layernorm(x, gamma, beta, o["y"], o["mean"], o["rstd"], stream=stream)
            wg.forge_layernorm_backward(dY, x, gamma, o["mean"], o["rstd"], o["dX"], o["dg"],
                                        o["db"], workspace=ws, stream=stream)

        run()
        sets.append((run, out, {k: v.clone() for k, v in out.items()}))
    torch.cuda.synchronize()

    def clear_and_compare(go):
        for _, out, _ in sets:
            for v in out.values():
                v.fill_(3.0)
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        for _, out, want in sets:
            assert all(torch.equal(out[k], want[k]) for k in want)

    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        clear_and_compare(lambda: [run(s) for s, (run, _, _) in zip(streams, sets)])
    graphs = []
    for run, _, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _ in range(4):
        clear_and_compare(lambda: [g.replay() for g in graphs])

    def side_by_side():
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()

    for _ in range(4):
        clear_and_compare(side_by_side)


def test_refused_tensors(env):
    torch, wg = env
    x, gamma, beta, dY = inputs(torch, 4, 64)
    y, s = torch.empty_like(x), torch.empty(4, device="cuda")
    with pytest.raises(TypeError):
        wg.forge_layernorm(x.half(), gamma, beta, y)
    with pytest.raises(TypeError):
        wg.forge_layernorm(x, gamma.bfloat16(), beta, y)
    with pytest.raises(TypeError):
        wg.forge_layernorm(x, None, beta, y)
    with pytest.raises(ValueError):
        wg.forge_layernorm(x.t(), gamma, beta, y)
    with pytest.raises(ValueError):
        wg.forge_layernorm(x, gamma[:32], beta, y)
    with pytest.raises(ValueError):
        wg.forge_layernorm(x, gamma, beta, y[:2])
    with pytest.raises(ValueError):
        wg.forge_layernorm(x, gamma, beta, y, s[:2])
    with pytest.raises(ValueError):
        wg.forge_layernorm(x, gamma.cpu(), beta, y)
    with pytest.raises(wg.ForgeError, match="ALIAS"):
        wg.forge_layernorm(x, gamma, beta, x)
    with pytest.raises(TypeError):
        wg.forge_layernorm_backward(dY, x, gamma, s, s, y.bfloat16(), gamma.clone())
    with pytest.raises(wg.ForgeError, match="SHAPE"):
        wg.forge_layernorm_backward(dY, x, gamma, s, s, y, gamma.clone(),
                                    workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert torch.isfinite(x).all()
