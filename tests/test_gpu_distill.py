"""Distillation from a teacher's top logits on the GPU against the formulas in
64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                  # half a float32 step, relative
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134}
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


def inputs(torch, T, V, K, zt="float32", ut="float32", it="int64", seed=0, ld=None, masked=True):
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    ld = (V + 7) // 8 * 8 if ld is None else ld
    u = torch.randn(T, K, generator=g, device="cuda") * 2 + 12
    ids = torch.randint(0, max(V, 1), (T, K), generator=g, device="cuda")
    z = torch.randn(T, ld, generator=g, device="cuda") * 2
    if V and K:
        z.scatter_reduce_(1, ids, u * 0.8, "amax")
    z[:, V:] = NAN                                  # columns that are not looked at
    weight = torch.rand(T, generator=g, device="cuda") + 0.5
    if masked and K:
        ids[torch.rand(T, K, generator=g, device="cuda") < 0.1] = -1
        ids[torch.rand(T, K, generator=g, device="cuda") < 0.05] = V
        weight[torch.rand(T, generator=g, device="cuda") < 0.15] = 0
    return (z.to(getattr(torch, zt)), u.to(getattr(torch, ut)), ids.to(getattr(torch, it)), weight, V)


def reference(torch, z, u, ids, weight, V, tau, scale, gt):
    """loss, grad, and how far float32 may be off each."""
    T, ld = z.shape
    K = u.shape[1]
    z64, u64, ids = z[:, :V].double(), u.double(), ids.long()
    w = torch.ones(T, device="cuda").double() if weight is None else weight.double()
    kept = (ids >= 0) & (ids < V) & (u64 != -INF)
    live = (w != 0) & kept.any(1) if K else torch.zeros(T, dtype=torch.bool, device="cuda")
    loss, grad = torch.zeros(T, device="cuda").double(), torch.zeros(T, ld, device="cuda").double()
    e_loss, e_grad = torch.zeros_like(loss), torch.zeros_like(grad)
    if V and K:
        at = torch.where(kept, ids, 0)
        logq = torch.log_softmax(torch.where(kept, u64 / tau, -INF), 1)
        zz = z64 / tau
        logp = zz - torch.logsumexp(zz, 1, keepdim=True)
        q = torch.where(kept, logq.exp(), 0)
        took = logp.gather(1, at)
        terms = torch.where(q > 0, q * (logq - took), 0)
        s = scale * w * tau * tau
        loss = torch.where(live, s * terms.sum(1), 0)
        p = logp.exp()
        target = torch.zeros_like(p).scatter_add_(1, at, q)
        c = (scale * w * tau)[:, None]
        grad[:, :V] = torch.where(live[:, None], c * (p - target), 0)
        # An exponential is off by 2 U (the instruction) and by its argument's error: the
        # difference to the maximum, its product with a rounded constant, 4 U of it.
        # A thread adds up to V / 512 terms of one sign one after the other (the loss
        # alone, 256 here), each addition off by up to U of what it has so far: on average
        # half of the sum and of random sign, 0.6 sqrt(256) = 10 U of the sum as a root mean
        # square, and threads' errors differ. 60 U are asked for; the teacher's as well.
        gap = (zz.amax(1, keepdim=True) - zz).clamp(max=1e30)
        gapu = torch.where(kept, (torch.where(kept, u64, -INF).amax(1, keepdim=True) - u64) / tau, 0)
        e_sum = (60 + 4 * (p * gap).sum(1, keepdim=True)) * U
        e_sumq = (60 + 4 * (q * gapu).sum(1, keepdim=True)) * U
        # v_exp_f32 and what follows flush what is below the normal numbers.
        e_p = p * (e_sum + (4 + 4 * gap) * U) + 2.0 ** -125
        e_q = q * (e_sumq + (4 + 4 * gapu) * U) + 2.0 ** -125
        e_t = torch.zeros_like(p).scatter_add_(1, at, torch.where(kept, e_q, 0)) + K * U * target
        value = c.abs() * (p + target)
        e_g = c.abs() * (e_p + e_t) + 4 * U * value
        e_grad[:, :V] = torch.where(live[:, None], e_g * (1 + HALF[gt]) + HALF[gt] * grad[:, :V].abs()
                                    + TINY[gt], 0)
        # loss / s = sum of q (du - dz) / tau, K + 6 roundings of its size and the error of
        # the q, plus the logarithms of the two sums (of at most log V, three roundings).
        apart = gapu + gap.gather(1, at)
        size = torch.where(q > 0, q * apart, 0).sum(1)
        drift = torch.where(q > 0, e_q * apart, 0).sum(1)
        logs = (e_sum + e_sumq)[:, 0] * 1.01 + 3 * U * (math.log(V + 1) + math.log(K + 1) + 1)
        e_loss = torch.where(live, s.abs() * ((K + 6) * U * size + drift + logs) + 4 * U * loss.abs(), 0)
    return loss, grad, e_loss, e_grad


def within(torch, got, want, tol, what):
    bad = ~(((got.double() - want).abs() <= tol) | (got.double() == want))
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(),
                           got[bad][:3].tolist(), want[bad][:3].tolist(), tol[bad][:3].tolist())


def check(torch, wg, args, gt="float32", tau=1.0, scale=1.0, in_place=False, **kw):
    z, u, ids, weight, V = args
    T, ld = z.shape
    loss = torch.full((T + 2,), 7.0, device="cuda")
    want = reference(torch, z, u, ids, weight, V, tau, scale, gt)
    alone = torch.empty(T, device="cuda")
    wg.forge_distill(z, u, ids, alone, vocab=V, weight=weight, temperature=tau, scale=scale, **kw)
    if in_place:
        grad = z
    else:
        big = torch.full((T * ld + 128,), 7.0, dtype=getattr(torch, gt), device="cuda")
        grad = big[64:64 + T * ld].view(T, ld)
    wg.forge_distill(z, u, ids, loss[1:-1], grad, vocab=V, weight=weight, temperature=tau, scale=scale,
                     **kw)
    within(torch, loss[1:-1], want[0], want[2], "loss")
    within(torch, grad, want[1], want[3], "grad")
    within(torch, alone, want[0], want[2], "loss alone")
    assert float(loss[0]) == float(loss[-1]) == 7.0
    if not in_place:
        assert bool((big[:64] == 7).all() and (big[64 + T * ld:] == 7).all())
    return loss[1:-1].clone(), grad


@pytest.mark.parametrize("T,V,K", [
    (1, 1, 1), (1, 8, 1), (2, 7, 3), (3, 100, 5), (5, 1000, 64), (4, 8192, 20), (3, 8193, 33),
    (2, 8191, 64), (2, 16384, 257), (7, 32003, 128), (3, 50021, 64), (2, 65536, 65), (2, 65537, 8),
    (2, 131072, 16), (1, 131073, 16), (2, 200001, 7), (33, 333, 100), (300, 2050, 17),
    (2, 5000, 1024), (64, 128256, 20)])
def test_sizes(env, T, V, K):
    torch, wg = env
    check(torch, wg, inputs(torch, T, V, K, seed=T))


@pytest.mark.parametrize("zt", list(HALF))
@pytest.mark.parametrize("gt", list(HALF))
@pytest.mark.parametrize("ut,it", [("float32", "int32"), ("bfloat16", "int64")])
@pytest.mark.parametrize("T,V,K,tau", [(5, 1003, 17, 1.0), (3, 20000, 40, 2.0), (290, 9001, 5, 0.5),
                                       (260, 40007, 12, 4.0)])
def test_types(env, T, V, K, tau, zt, gt, ut, it):
    torch, wg = env
    check(torch, wg, inputs(torch, T, V, K, zt, ut, it, seed=V), gt, tau, scale=1.0 / T)


# Every thread of either path with all the entries it can have.
@pytest.mark.parametrize("zt", list(HALF))
@pytest.mark.parametrize("T,V,K", [(2, 40000, 1024), (3, 200001, 1000), (1, 17000, 1023), (70, 40000, 1024),
                                   (70, 5000, 769), (200, 140000, 1022)])
def test_the_most_entries(env, T, V, K, zt):
    torch, wg = env
    check(torch, wg, inputs(torch, T, V, K, zt, "bfloat16", "int32", seed=14), "bfloat16", 1.5, 0.5)


@pytest.mark.parametrize("zt", list(HALF))
@pytest.mark.parametrize("T,V,K", [(5, 1003, 17), (3, 20000, 40), (290, 9001, 5), (270, 131072, 9),
                                   (300, 70001, 3), (2, 140000, 20)])
def test_gradient_in_place(env, T, V, K, zt):
    torch, wg = env
    args = inputs(torch, T, V, K, zt, seed=4)
    _, apart = check(torch, wg, args, zt, 1.5)
    _, same = check(torch, wg, args, zt, 1.5, in_place=True)
    assert torch.equal(apart, same)


@pytest.mark.parametrize("T,V,K,zt", [(600, 3000, 30, "bfloat16"), (600, 40000, 64, "bfloat16"),
                                      (520, 128256, 64, "bfloat16"), (400, 50021, 32, "float32"),
                                      (9000, 1001, 3, "float32"), (300, 262144, 4, "bfloat16"),
                                      (1100, 65537, 10, "bfloat16")])
def test_many_rows(env, T, V, K, zt):
    torch, wg = env
    check(torch, wg, inputs(torch, T, V, K, zt, "bfloat16", "int32", seed=6), "bfloat16", 2.0, 1.0 / T)


def test_more_items_than_workgroups(env):
    torch, wg = env
    T = (1 << 20) + 700
    check(torch, wg, inputs(torch, T, 24, 2, "bfloat16", seed=2), "bfloat16")


def test_padded_columns(env):
    """A pitch wider than the vocabulary, by whole chunks too."""
    torch, wg = env
    for V, ld in ((1000, 1024), (3, 64), (8192, 16400), (8190, 8192), (5000, 30000)):
        for T in (3, 400):
            _, grad = check(torch, wg, inputs(torch, T, V, 9, "bfloat16", ld=ld), "bfloat16")
            assert (grad[:, V:] == 0).all()


@pytest.mark.parametrize("zt,gt", [("bfloat16", "bfloat16"), ("float32", "bfloat16"), ("float32", "float32")])
@pytest.mark.parametrize("V,ld", [(17000, 40000), (20480, 24576), (20481, 20488), (33000, 33016), (70001, 100000)])
def test_padded_columns_of_few_rows(env, V, ld, zt, gt):
    """Chunks that lie past the vocabulary, in part or as a whole; into the logits too."""
    torch, wg = env
    args = inputs(torch, 3, V, 9, zt, ld=ld, seed=4)
    _, grad = check(torch, wg, args, gt)
    assert (grad[:, V:] == 0).all()
    if zt == gt:
        check(torch, wg, args, gt, in_place=True)


@pytest.mark.parametrize("T", [8, 70])
def test_rows_of_a_large_vocabulary_left_out_or_masked(env, T):
    """The loss alone too is cut into chunks, or not, at this vocabulary."""
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, T, 70000, 10, masked=False)
    weight[0] = 0
    ids[1] = -1
    u[2] = -INF
    z[0, 5] = NAN
    z[1] = INF
    z[2] = -INF
    keep = z.gather(1, ids.clamp(min=0))
    z[3, : V // 2] = -INF
    z[4, 100:] = -INF
    z[5] = torch.finfo(torch.float32).min
    z.scatter_(1, ids.clamp(min=0), keep)
    ids[6, 1:] = ids[6, 0]
    u[6, 2:] = -INF
    loss, grad = check(torch, wg, (z, u, ids, weight, V))
    assert (loss[:3] == 0).all() and (grad[:3] == 0).all() and torch.isfinite(loss).all()
    loss, grad = torch.full((T,), 5.0, device="cuda"), torch.full((T, V), 5.0, device="cuda")
    none = u[:, :0].contiguous(), ids[:, :0].contiguous()
    wg.forge_distill(z, *none, loss, grad, weight=weight)
    assert (loss == 0).all() and (grad == 0).all()
    wg.forge_distill(z, *none, loss.fill_(5.0), weight=weight)
    assert (loss == 0).all()


@pytest.mark.parametrize("T", [4, 300])
def test_an_id_that_recurs(env, T):
    torch, wg = env
    for K in (2, 70, 300):
        z, u, ids, weight, V = inputs(torch, T, 9000, K, masked=False)
        ids[:, 1:] = ids[:, :1]
        check(torch, wg, (z, u, ids, weight, V))
        ids[:, ::2] = 3
        check(torch, wg, (z, u, ids, weight, V))


@pytest.mark.parametrize("T", [12, 300])
def test_rows_that_are_left_out(env, T):
    """Weight 0, no entry with an id, no entry with a logit: loss 0 and zeros, whatever the logits."""
    torch, wg = env
    for V in (1000, 20000):
        z, u, ids, weight, V = inputs(torch, T, V, 10, masked=False)
        weight[0] = 0
        ids[1] = -1
        ids[2] = V
        u[3] = -INF
        ids[4] = 1 << 40                             # does not become an id in 32 bits
        z[0, 5] = NAN
        z[1] = INF
        z[2] = NAN
        z[3] = -INF
        u[0], u[1] = NAN, NAN
        loss, grad = check(torch, wg, (z, u, ids, weight, V))
        assert (loss[:5] == 0).all() and (grad[:5] == 0).all()
        # not left out (below 0 is possible where an id recurs: each entry has its own log q)
        assert (loss[5:] != 0).all() and torch.isfinite(loss).all()


@pytest.mark.parametrize("T", [8, 300])
def test_masked_columns(env, T):
    """Columns of -infinity and of the type's lowest value; entries of -infinity."""
    torch, wg = env
    for V in (1000, 20000):
        z, u, ids, weight, V = inputs(torch, T, V, 6, masked=False)
        keep = z.gather(1, ids)
        z[:, ::2] = -INF
        z[1, :] = torch.finfo(torch.float32).min
        z[2, : V // 2] = -INF
        z.scatter_(1, ids, keep)
        u[3, 1:] = -INF
        u[4, :3] = -INF
        check(torch, wg, (z, u, ids, weight, V))
        # a teacher's column that the student has masked: an infinite loss, a finite gradient
        z[5, ids[5, 0]] = -INF
        loss, grad = check(torch, wg, (z, u, ids, weight, V))
        assert float(loss[5]) == INF and torch.isfinite(grad[:, :V]).all()


@pytest.mark.parametrize("T", [8, 300])
def test_a_row_that_is_not_finite_stays_alone(env, T):
    torch, wg = env
    for V in (1000, 20000):
        z, u, ids, weight, V = inputs(torch, T, V, 6, masked=False)
        loss, grad = check(torch, wg, (z, u, ids, weight, V))
        z[1, V - 1] = NAN
        z[2, 0] = INF
        z[3, :V] = -INF
        u[4, 2] = NAN
        u[5, 1] = INF
        l2, g2 = torch.empty_like(loss), torch.empty_like(grad)
        wg.forge_distill(z, u, ids, l2, g2, vocab=V, weight=weight)
        assert torch.isnan(l2[1:6]).all()
        assert torch.isnan(g2[1:4, :V]).any(1).all()
        for k in (4, 5):
            assert torch.isnan(g2[k][ids[k]]).any()
        rest = [0] + list(range(6, T))
        assert torch.equal(l2[rest], loss[rest]) and torch.equal(g2[rest], grad[rest])


@pytest.mark.parametrize("T", [3, 300])
def test_logits_far_below_zero(env, T):
    """Threads, waves and chunks whose columns are all masked beside logits of -900."""
    torch, wg = env
    for V in (700, 9000, 50000):
        z, u, ids, weight, V = inputs(torch, T, V, 6, masked=False)
        z[:, :V] -= 900
        keep = z.gather(1, ids)
        z[0, : V // 2] = -INF
        z[1, V // 3:V] = -INF
        z[2, 64:] = -INF
        z.scatter_(1, ids, keep)
        check(torch, wg, (z, u, ids, weight, V))


def test_far_logits(env):
    """A student that is sure, and temperatures far from 1."""
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, 6, 3000, 8, masked=False)
    z[0, 17] = 300.0
    z[1] *= 100
    z[2] = 5.0
    for tau in (0.05, 1.0, 30.0):
        check(torch, wg, (z, u, ids, weight, V), tau=tau)
    check(torch, wg, (z, u, ids, None, V), scale=-2.0)
    check(torch, wg, (z, u, ids, weight, V), scale=0.0)


def test_no_rows_columns_or_entries(env):
    torch, wg = env
    for T, V, K in ((0, 10, 3), (3, 0, 2), (3, 10, 0)):
        z, u, ids, weight, V = inputs(torch, T, V, K, ld=16, masked=False)
        loss, grad = torch.full((T,), 5.0, device="cuda"), torch.full((T, 16), 5.0, device="cuda")
        wg.forge_distill(z, u, ids, loss, grad, vocab=V, weight=weight)
        assert (loss == 0).all() and (grad == 0).all()
        wg.forge_distill(z, u, ids, loss, vocab=V)
        assert (loss == 0).all()


def test_shapes(env):
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, 12, 1000, 5)
    loss, grad = check(torch, wg, (z, u, ids, weight, V))
    l2, g2 = torch.empty(3, 4, device="cuda"), torch.empty(3, 4, 1000, device="cuda")
    wg.forge_distill(z.view(3, 4, -1), u.view(3, 4, 5), ids.view(3, 4, 5), l2, g2,
                     weight=weight.view(3, 4))
    assert torch.equal(l2.view(-1), loss) and torch.equal(g2.view(12, -1), grad)
    l1, g1 = torch.empty((), device="cuda"), torch.empty(1000, device="cuda")
    row = int(torch.nonzero(weight)[0])
    wg.forge_distill(z[row], u[row], ids[row], l1, g1, weight=weight[row])
    assert float(l1) == float(loss[row]) and torch.equal(g1, grad[row])


@pytest.mark.parametrize("T,V,K,tau", [(7, 3001, 20, 1.0), (260, 9000, 5, 2.0)])
def test_differences(env, T, V, K, tau):
    """The gradient against differences of the loss along a direction."""
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, T, V, K)
    z[:, V:] = 0
    args = (z, u, ids, weight, V)
    loss, grad = check(torch, wg, args, tau=tau)
    g = torch.Generator(device="cuda").manual_seed(8)
    step = torch.randn(z.shape, generator=g, device="cuda")
    h = 2.0 ** -7
    side, side64, noise = [], [], 0.0
    for s in (1, -1):
        moved = z + s * h * step
        out = torch.empty_like(loss)
        wg.forge_distill(moved, u, ids, out, vocab=V, weight=weight, temperature=tau)
        want = reference(torch, moved, u, ids, weight, V, tau, 1.0, "float32")
        side.append(float(out.double().sum()))
        side64.append(float(want[0].sum()))
        noise += float(want[2].sum() + U * (moved.double().abs() * want[1].abs()).sum())
    slope, slope64 = (side[0] - side[1]) / (2 * h), (side64[0] - side64[1]) / (2 * h)
    assert abs(slope - slope64) <= noise / (2 * h)
    # The error of a difference of this width: a third derivative times h^2 / 6.
    w = h / 16
    near = [float(reference(torch, z.double() + s * w * step.double(), u, ids, weight, V, tau, 1.0,
                            "float32")[0].sum()) for s in (1, -1)]
    bend = abs((near[0] - near[1]) / (2 * w) - slope64) * 1.01
    want = reference(torch, *args, tau, 1.0, "float32")
    along = float((grad.double() * step.double()).sum())
    assert abs(slope - along) <= noise / (2 * h) + bend + float((want[3] * step.abs()).sum())


def test_the_same_bits_again(env):
    torch, wg = env
    for T, V in ((9, 50021), (700, 30000)):
        args = inputs(torch, T, V, 40, "bfloat16")
        first = check(torch, wg, args, "bfloat16")
        for _ in range(2):
            ws = torch.randint(0, 255, (wg.library().forge_distill_workspace(T, V, 40),),
                               dtype=torch.uint8, device="cuda")
            again = check(torch, wg, args, "bfloat16", workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("T,V", [(6, 40000), (300, 9000)])
def test_captured_and_two_streams(env, T, V):
    torch, wg = env
    sets = []
    for seed in (1, 2):
        z, u, ids, weight, V = inputs(torch, T, V, 33, "bfloat16", seed=seed)
        loss, grad = torch.empty(T, device="cuda"), torch.empty_like(z)
        ws = torch.empty(wg.library().forge_distill_workspace(T, V, 33), dtype=torch.uint8, device="cuda")

        def run(stream=None, a=(z, u, ids, loss, grad), k=dict(vocab=V, weight=weight, workspace=ws)):
            wg.forge_distill(*a, stream=stream, **k)

        run()
        sets.append((run, (loss, grad), (loss.clone(), grad.clone())))
    torch.cuda.synchronize()

    def clear_and_compare(go):
        for _, out, _ in sets:
            for v in out:
                v.fill_(3.0)
        torch.cuda.synchronize()
        go()
        torch.cuda.synchronize()
        for _, out, want in sets:
            assert all(torch.equal(a, b) for a, b in zip(out, want))

    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        clear_and_compare(lambda: [run(s) for s, (run, _, _) in zip(streams, sets)])
    graphs = []
    for run, _, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)

    def side_by_side():
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()

    for _ in range(4):
        clear_and_compare(lambda: [g.replay() for g in graphs])
        clear_and_compare(side_by_side)


def test_offsets_beyond_32_bits(env):
    """The last rows of logits of more than 2^32 bytes."""
    torch, wg = env
    T, V = 17000, 131072
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    z[-3:] = torch.randn(3, V, generator=g, device="cuda").to(torch.bfloat16)
    u = torch.randn(T, 4, generator=g, device="cuda")
    ids = torch.randint(0, V, (T, 4), generator=g, device="cuda")
    weight = torch.zeros(T, device="cuda")
    weight[-3:] = 1
    loss = torch.empty(T, device="cuda")
    want = reference(torch, z[-3:].clone(), u[-3:], ids[-3:], weight[-3:], V, 1.0, 1.0, "bfloat16")
    wg.forge_distill(z, u, ids, loss, z, weight=weight)
    within(torch, loss[-3:], want[0], want[2], "loss")
    within(torch, z[-3:], want[1], want[3], "grad")
    assert not loss[:-3].any() and not z[:-3].any()


def test_refused_tensors(env):
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, 4, 64, 3)
    loss, grad = torch.empty(4, device="cuda"), torch.empty_like(z)
    call = wg.forge_distill
    for bad in (dict(logits=z.half()), dict(teacher=u.half()), dict(ids=ids.short()), dict(loss=None),
                dict(loss=loss.double()), dict(grad=grad.half()), dict(weight=weight.bfloat16())):
        with pytest.raises(TypeError):
            call(**{**dict(logits=z, teacher=u, ids=ids, loss=loss, grad=grad, weight=weight), **bad})
    for bad in (dict(teacher=u[:, :2]), dict(ids=ids[:3]), dict(loss=loss[:2]), dict(grad=grad[:, :32]),
                dict(weight=weight[:1]), dict(logits=z.t()), dict(ids=ids.cpu())):
        with pytest.raises(ValueError):
            call(**{**dict(logits=z, teacher=u, ids=ids, loss=loss, grad=grad, weight=weight), **bad})
    for bad, name in ((dict(vocab=65), "SHAPE"), (dict(vocab=-1), "SHAPE"), (dict(temperature=0.0), "HPARAM"),
                      (dict(scale=math.nan), "HPARAM"), (dict(grad=z[:4]), None)):
        kw = {**dict(logits=z, teacher=u, ids=ids, loss=loss, grad=grad, weight=weight), **bad}
        if name is None:
            call(**kw)                               # in place
        else:
            with pytest.raises(wg.ForgeError, match=name):
                call(**kw)
    with pytest.raises(wg.ForgeError, match="SHAPE"):
        call(z, u, ids, loss, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("byte", [0, 0x7F, 0xFF])
@pytest.mark.parametrize("T,V", [(4, 40000), (40, 70000), (300, 9000)])
def test_what_the_workspace_holds_means_nothing(env, T, V, byte):
    """Zeros, large numbers or NaN there, with rows of weight 0 and entries that are not there."""
    torch, wg = env
    z, u, ids, weight, V = inputs(torch, T, V, 30, seed=5)
    weight[1], weight[2] = 0, 1
    ids[2, 1:] = -1
    ws = torch.full((1 << 20,), byte, dtype=torch.uint8, device="cuda")
    loss, grad = check(torch, wg, (z, u, ids, weight, V), "bfloat16", workspace=ws)
    assert float(loss[1]) == 0 and not grad[1].any()
    l2, g2 = torch.empty_like(loss), torch.empty_like(grad)
    wg.forge_distill(z, u, ids, l2, g2, vocab=V, weight=weight)
    assert torch.equal(loss, l2) and torch.equal(grad, g2)
