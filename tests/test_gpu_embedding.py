"""Embedding lookup and gradient on the GPU against the formulas in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                  # half a float32 step, relative
ADAM = dict(step=7, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SGDM = dict(lr=1e-2, momentum=0.9, weight_decay=1e-2)

# T, V, d and how the ids fall
CASES = [
    (1, 1, 8, "uniform"), (1, 100, 64, "uniform"), (0, 5, 64, "uniform"), (3, 1, 8, "uniform"),
    (31, 7, 24, "uniform"), (32, 1, 40, "one"), (33, 2, 256, "one"), (64, 3, 1032, "one"),
    (1000, 513, 72, "zipf"), (1021, 5003, 512, "zipf"), (2000, 50, 2056, "zipf"),
    (4096, 131072, 16, "uniform"), (4096, 300000, 8, "uniform"), (5000, 4000000, 8, "spread"),
    (16384, 1000, 64, "zipf"), (16385, 1000, 64, "zipf"), (16384, 513, 8, "one"),
    (20000, 77, 128, "one"), (50001, 128256, 32, "zipf"), (70000, 70000, 16, "sorted"),
    (70000, 70000, 16, "reversed"), (300, 40, 4104, "none"), (40000, 600000, 8, "spread"),
    (65536, 300, 8, "zipf"), (65537, 128256, 8, "zipf"), (262144, 5000, 8, "zipf"),
    (262145, 128256, 8, "zipf"), (1000003, 999983, 8, "zipf"), (4097, 600, 64, "zipf"),
    (1024, 900, 512, "one"), (1024, 3, 1032, "zipf"), (1025, 3, 1032, "zipf"), (900, 1, 4104, "one"),
    (777, 5000, 24, "zipf"), (255, 5000, 24, "zipf"), (256, 70, 1032, "zipf"), (256, 900, 512, "one"),
    (257, 900, 512, "one"), (256, 200000, 16, "uniform"), (100, 1000, 4104, "zipf"),
]


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


def make_ids(torch, T, V, how, dtype, seed=3):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(T, generator=g, dtype=torch.float64)
    if how == "zipf":
        ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    elif how == "one":
        ids = torch.full((T,), V - 1)
    elif how == "sorted":
        ids = torch.arange(T) % V
    elif how == "reversed":
        ids = V - 1 - torch.arange(T) % V
    elif how == "none":
        ids = torch.full((T,), -1)
    else:
        ids = (u * V).long().clamp(0, V - 1)
    if how in ("zipf", "uniform", "spread") and T > 8:      # nobody's ids, at both ends
        far = [-1, V, -(1 << 31), (1 << 31) - 1]
        if dtype == torch.int64:
            far += [1 << 32, -(1 << 62), (1 << 62) + 1]
        ids[torch.arange(0, T, 7)[: len(far)]] = torch.tensor(far[: len(range(0, T, 7))])
    return ids.to(dtype)


def grad64(torch, ids, dY, V, scale):
    """The gradient in float64 and a bound of the float32 sums' error."""
    ids, dY = ids.cpu().long(), dY.cpu().double()
    ok = (ids >= 0) & (ids < V)
    g = torch.zeros(V, dY.shape[1], dtype=torch.float64)
    a = torch.zeros_like(g)
    n = torch.zeros(V, 1, dtype=torch.float64)
    s = float(torch.tensor(scale, dtype=torch.float32))
    g.index_add_(0, ids[ok], dY[ok] * s)
    a.index_add_(0, ids[ok], dY[ok].abs() * abs(s))
    n.index_add_(0, ids[ok], torch.ones(int(ok.sum()), 1, dtype=torch.float64))
    # A term passes at most n additions, each off by half a step of a partial sum that the
    # magnitudes bound, and one product.
    return g, (n + 1) * U * a, n


@pytest.mark.parametrize("ids_t", ["int32", "int64"])
@pytest.mark.parametrize("types", ["f32-f32", "f32-bf16", "bf16-f32", "bf16-bf16"])
@pytest.mark.parametrize("T,V,d", [(1, 1, 8), (8, 1000, 64), (1, 777, 4096), (1000, 50, 520),
                                   (257, 300, 2056), (33, 9, 24)])
def test_lookup(env, T, V, d, types, ids_t):
    torch, wg = env
    tt, ot = ({"f32": torch.float32, "bf16": torch.bfloat16}[k] for k in types.split("-"))
    table = torch.randn(V, d, device="cuda").to(tt)
    ids = make_ids(torch, T, V, "uniform", getattr(torch, ids_t))
    out = torch.full((T, d), 7.0, device="cuda", dtype=ot)
    scale = math.sqrt(d)
    wg.forge_embedding(table, ids.cuda(), out, scale=scale)
    i = ids.long()
    ok = (i >= 0) & (i < V)
    want = torch.zeros(T, d)
    want[ok] = table.cpu().float()[i[ok]] * torch.tensor(scale, dtype=torch.float32)
    assert torch.equal(out.cpu(), want.to(ot))          # one product, one rounding: the same bits


def test_lookup_keeps_nonfinite_and_other_rows(env):
    torch, wg = env
    table = torch.tensor([[math.inf] * 8, [math.nan] * 8, [1.0] * 8], device="cuda")
    ids = torch.tensor([[2, 0], [1, -1]], device="cuda")
    out = torch.full((3, 2, 8), 5.0, device="cuda")
    wg.forge_embedding(table, ids, out[:2], scale=0.5)
    got = out.cpu()
    assert bool((got[0, 0] == 0.5).all()) and bool(torch.isinf(got[0, 1]).all())
    assert bool(torch.isnan(got[1, 0]).all()) and bool((got[1, 1] == 0).all())
    assert bool((got[2] == 5.0).all())


@pytest.mark.parametrize("dy", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,d,how", CASES)
def test_gradient(env, T, V, d, how, dy):
    torch, wg = env
    ids = make_ids(torch, T, V, how, torch.int64 if dy == "bf16" else torch.int32)
    dY = torch.randn(T, d).to(torch.bfloat16 if dy == "bf16" else torch.float32)
    want, tol, n = grad64(torch, ids, dY, V, 1.7)
    grad = torch.full((V, d), 9.0, device="cuda")
    wg.forge_embedding_grad(ids.cuda(), dY.cuda(), grad, scale=1.7)
    got = grad.double().cpu()
    assert bool(((got - want).abs() <= tol).all())
    assert bool((got[n[:, 0] == 0] == 0).all())
    # accumulated: one more rounding, rows without a token untouched
    base = torch.randn(V, d)
    acc = base.cuda()
    wg.forge_embedding_grad(ids.cuda(), dY.cuda(), acc, scale=1.7, accumulate=True)
    has = n[:, 0] > 0
    assert torch.equal(acc.cpu()[~has], base[~has])
    assert torch.equal(acc.cpu()[has], (base + grad.cpu())[has])
    again = torch.empty_like(grad)
    wg.forge_embedding_grad(ids.cuda(), dY.cuda(), again, scale=1.7)
    assert torch.equal(again, grad)


@pytest.mark.parametrize("T,V,d,how", [c for c in CASES if c[1] * c[2] < 3e6])
def test_fused_steps_are_the_gradient_and_the_step(env, T, V, d, how):
    torch, wg = env
    ids = make_ids(torch, T, V, how, torch.int64).cuda()
    dY = (torch.randn(T, d) * 0.1).to(torch.bfloat16).cuda()
    W, m = torch.randn(V, d, device="cuda"), torch.randn(V, d, device="cuda") * 0.1
    v = torch.rand(V, d, device="cuda") * 0.01
    grad = torch.empty(V, d, device="cuda")
    wg.forge_embedding_grad(ids, dY, grad, scale=0.3)
    for eps in (1e-8, 0.0):
        st, ref = ([t.clone() for t in (W, m, v)] for _ in range(2))
        hp = dict(ADAM, eps=eps)
        wg.forge_embedding_adamw(ids, dY, *st, scale=0.3, **hp)
        wg.forge_adamw(grad, *ref, **hp)
        assert all(torch.equal(a, b) for a, b in zip(st, ref))
    st, ref = ([t.clone() for t in (W, m)] for _ in range(2))
    wg.forge_embedding_sgdm(ids, dY, *st, scale=0.3, **SGDM)
    wg.forge_sgdm(grad, *ref, **SGDM)
    assert all(torch.equal(a, b) for a, b in zip(st, ref))


def test_fused_adamw_against_64_bits(env):
    torch, wg = env
    T, V, d = 3000, 701, 136
    ids = make_ids(torch, T, V, "zipf", torch.int64)
    dY = torch.randn(T, d)
    W, m, v = torch.randn(V, d), torch.randn(V, d), torch.rand(V, d) + 0.5
    g, tg, _ = grad64(torch, ids, dY, V, 1.0)
    st = [t.clone().cuda() for t in (W, m, v)]
    wg.forge_embedding_adamw(ids.cuda(), dY.cuda(), *st, **ADAM)
    b1, b2, lr = ADAM["beta1"], ADAM["beta2"], ADAM["lr"]
    m1 = b1 * m.double() + (1 - b1) * g
    v1 = b2 * v.double() + (1 - b2) * g * g
    den = (v1 / (1 - b2 ** ADAM["step"])).sqrt() + ADAM["eps"]
    s = lr / (1 - b1 ** ADAM["step"])
    w1 = W.double() * (1 - lr * ADAM["weight_decay"]) - s * m1 / den
    # The roundings of the step (see test_gpu_clip), and what the gradient's error adds: linear in
    # m, 2 g tg in v, and through both in the update.
    tm = 4 * U * (abs(b1 * m.double()) + abs((1 - b1) * g)) + (1 - b1) * tg
    dv = (1 - b2) * (2 * abs(g) * tg + tg * tg)
    tv = 6 * U * v1 + dv
    tw = 4 * U * abs(w1) + 4 * U * abs(W.double()) + s / den * (tm + abs(m1) * (16 * U + dv / v1))
    for got, want, tol in zip(st, (w1, m1, v1), (tw, tm, tv)):
        assert bool(((got.double().cpu() - want).abs() <= tol).all())


def test_gradient_against_differences(env):
    """The lookup's loss is linear in the table, so its gradient is the
    difference of two losses exactly, up to the rounding of the sums."""
    torch, wg = env
    T, V, d = 200, 17, 16
    ids = make_ids(torch, T, V, "zipf", torch.int64).cuda()
    dY = torch.randn(T, d, device="cuda")
    table = torch.randn(V, d, device="cuda")
    grad = torch.empty(V, d, device="cuda")
    wg.forge_embedding_grad(ids, dY, grad, scale=2.0)

    def loss(t):
        out = torch.empty(T, d, device="cuda")
        wg.forge_embedding(t, ids, out, scale=2.0)
        return (out.double() * dY.double()).sum()

    for r, c in ((0, 0), (1, 5), (16, 15), (3, 9)):
        up, down = table.clone(), table.clone()
        up[r, c] += 0.5
        down[r, c] -= 0.5
        step = float(up[r, c].double() - down[r, c].double())
        diff = float(loss(up) - loss(down)) / step
        # the lookup's products by 2 are exact; the sum of at most T terms of the gradient is not
        size = float((dY.double()[:, c].abs() * (ids == r)).sum()) * 2
        assert abs(diff - float(grad[r, c])) <= (T + 1) * U * size + 1e-9


def test_nonfinite_tokens_stay_in_their_rows(env):
    torch, wg = env
    ids = torch.tensor([0, 1, 2, -1, 1], device="cuda")
    dY = torch.ones(5, 8, device="cuda")
    dY[1, 3], dY[3, :] = math.inf, math.nan             # row 3 is nobody's
    grad = torch.empty(3, 8, device="cuda")
    wg.forge_embedding_grad(ids, dY, grad)
    want = torch.tensor([[1.0] * 8, [2.0] * 8, [1.0] * 8])
    want[1, 3] = math.inf
    assert torch.equal(grad.cpu(), want)


def test_graph_and_streams(env):
    torch, wg = env
    for T, V in ((700, 90), (30000, 90)):
        d = 64
        ids = make_ids(torch, T, V, "zipf", torch.int64).cuda()
        dY = torch.randn(T, d, device="cuda")
        W, b = torch.randn(V, d, device="cuda"), torch.zeros(V, d, device="cuda")
        rW, rb = W.clone(), b.clone()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            wg.forge_embedding_sgdm(ids, dY, W, b, **SGDM)
        for k in range(4):
            ids.copy_(make_ids(torch, T, V, "zipf", torch.int64, seed=50 + k).cuda())
            dY.mul_(-1.25)
            graph.replay()
            torch.cuda.synchronize()
            wg.forge_embedding_sgdm(ids, dY, rW, rb, **SGDM)
            torch.cuda.synchronize()
            assert torch.equal(W, rW) and torch.equal(b, rb), k
        side = torch.cuda.Stream()
        one, two = torch.empty(V, d, device="cuda"), torch.empty(V, d, device="cuda")
        torch.cuda.synchronize()
        wg.forge_embedding_grad(ids, dY, one, stream=side)
        wg.forge_embedding_grad(ids, dY, two)
        torch.cuda.synchronize()
        assert torch.equal(one, two)


def test_binding_refuses(env):
    torch, wg = env
    table = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    out = torch.zeros(3, 8, device="cuda")
    with pytest.raises(TypeError, match="int32 or int64"):
        wg.forge_embedding(table, ids.to(torch.int16), out)
    with pytest.raises(ValueError, match="shape"):
        wg.forge_embedding(table, ids, out[:2])
    with pytest.raises(ValueError, match="on the GPU"):
        wg.forge_embedding(table, ids.cpu(), out)
    with pytest.raises(TypeError, match="float32"):
        wg.forge_embedding_grad(ids, out, table.to(torch.bfloat16))
    with pytest.raises(wg.ForgeError, match="SHAPE"):
        wg.forge_embedding_grad(ids, out, table,
                                workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(wg.ForgeError, match="SHAPE"):                # 2^22 rows are the most
        wg.forge_embedding_grad(ids, out, torch.empty((1 << 22) + 1, 8, device="cuda"))
    with pytest.raises(wg.ForgeError, match="HPARAM"):
        wg.forge_embedding(table, ids, out, scale=math.nan)
    with pytest.raises(wg.ForgeError, match="ALIGN"):
        wg.forge_embedding(torch.zeros(4, 4, device="cuda"), ids, torch.zeros(3, 4, device="cuda"))
    with pytest.raises(wg.ForgeError, match="CLIP"):
        wg.forge_embedding_adamw(ids, out, table, table.clone(), table.clone(), step=1,
                                 max_grad_norm=1.0)
    assert bool((table == 0).all())


def test_lookup_in_an_empty_table(env):
    torch, wg = env
    out = torch.full((3, 8), 5.0, device="cuda")
    ids = torch.tensor([0, -1, 4], device="cuda")
    wg.forge_embedding(torch.empty(0, 8, device="cuda"), ids, out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("types", ["f32-f32", "f32-bf16", "bf16-f32", "bf16-bf16"])
def test_lookup_of_an_output_past_the_cache(env, types):
    torch, wg = env
    tt, ot = ({"f32": torch.float32, "bf16": torch.bfloat16}[k] for k in types.split("-"))
    T, V, d = (1 << 27) // 1032 // (4 if ot == torch.float32 else 2) + 1, 50, 1032
    table = torch.randn(V, d, device="cuda").to(tt)
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % (V + 1)
    out = torch.empty(T, d, device="cuda", dtype=ot)
    wg.forge_embedding(table, ids, out, scale=3.0)
    want = torch.cat([table.float() * 3.0, torch.zeros(1, d, device="cuda")]).to(ot)
    assert torch.equal(out, want[ids.long()])


def test_outputs_of_more_workgroups_than_a_launch(env):
    """2^22 rows of 1026 units: beyond 2^32 units and 2^22 workgroups (also with four pieces to
    one), so that every kernel goes round its loop and the row of a unit takes 64 bits."""
    torch, wg = env
    V, d, part = 1 << 22, 4104, 1 << 18
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("69 GB of output and its comparison do not fit")
    big = torch.empty(V, d, device="cuda")
    # Rows at both ends and around places 2^22 workgroups and 2^32 units in.
    rows = [0, 1, V - 1, V - 2, *((p // 1026 + k) for p in (1 << 30, 1 << 32) for k in (-2, -1, 0, 1, 2))]
    assert all(0 <= r < V for r in rows)
    for T in (200, 300):                    # looked through, and sorted
        ids = torch.tensor([rows[k % len(rows)] for k in range(T)], device="cuda")
        dY = torch.randn(T, d, device="cuda")
        small = torch.unique(ids)           # the same gradient over the rows with tokens alone
        want = torch.empty(len(small), d, device="cuda")
        wg.forge_embedding_grad(torch.searchsorted(small, ids), dY, want, scale=1.5)
        big.fill_(7.0)
        wg.forge_embedding_grad(ids, dY, big, scale=1.5)
        assert torch.equal(big[small], want)
        wg.forge_embedding_grad(ids, dY, big, scale=1.5, accumulate=True)
        assert torch.equal(big[small], want + want)
        big[small] = 0
        assert not any(bool(big[r:r + part].any()) for r in range(0, V, part))
    table = torch.randn(37, 2 * d, device="cuda")
    ids = torch.arange(V, device="cuda", dtype=torch.int32) % 38          # one of them nobody's
    out = big.view(torch.bfloat16)
    wg.forge_embedding(table, ids, out, scale=3.0)
    want = torch.cat([table * 3.0, torch.zeros(1, 2 * d, device="cuda")]).to(torch.bfloat16)
    for r in range(0, V, part // 4):
        assert torch.equal(out[r:r + part // 4], want[ids[r:r + part // 4].long()]), r
    del big, out
    torch.cuda.empty_cache()
