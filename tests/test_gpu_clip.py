"""Global gradient norm and clipped steps on the GPU against the formulas in
64 bits, and bitwise against the unclipped elementwise steps."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                  # half a float32 step, relative
ADAM = dict(step=3, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SGDM = dict(lr=1e-2, momentum=0.9, weight_decay=1e-2)

LISTS = {
    "one": [1],
    "empty": [],
    "zeros": [0, 0],
    "odd": [1, 2, 3, 5, 7, 8, 9, 0, 4095, 4096, 4097],
    "chunk edges": [16383, 16384, 16385, 8191, 32768],
    "many": [1 + (k * 7919) % 3001 for k in range(300)],
    "large": [3_000_001, 5, 1_000_000],
}


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


def make(torch, sizes, dtypes, seed, std=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kinds = {"f32": [torch.float32], "bf16": [torch.bfloat16],
             "both": [torch.float32, torch.bfloat16]}[dtypes]

    def randn(n):
        return torch.randn(n, generator=g, device="cuda") * std

    grads = [randn(n).to(kinds[k % len(kinds)]) for k, n in enumerate(sizes)]
    W, m = [randn(n) for n in sizes], [randn(n) * 0.1 for n in sizes]
    v = [randn(n) ** 2 + 1e-6 for n in sizes]
    return grads, W, m, v


def norm64(grads):
    s = sum(float((g.double().cpu() ** 2).sum()) for g in grads)
    return math.sqrt(s)


def check_norm(out, ref, max_norm):
    # The sums are float64 (their error is far below float32's), each result is rounded once.
    n, c = (float(x) for x in out.double().cpu())
    coef = min(1.0, max_norm / (ref + 1e-6))
    assert abs(n - ref) <= ref * U * 1.001, (n, ref)
    assert abs(c - coef) <= coef * U * 1.001, (c, coef)


@pytest.mark.parametrize("dtypes", ["f32", "bf16", "both"])
@pytest.mark.parametrize("name", list(LISTS))
def test_norm(env, name, dtypes):
    torch, wg = env
    grads, *_ = make(torch, LISTS[name], dtypes, 11)
    ref = norm64(grads)
    for max_norm in (0.5 * ref, 2 * ref, 0.0, math.inf):
        out = torch.full((2,), -7.0, device="cuda")
        wg.forge_grad_norm(wg.ForgeTensorList(grads), out, max_norm=max_norm)
        check_norm(out, ref, max_norm)


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-44, 0.0])
def test_norm_over_the_whole_range(env, value):
    torch, wg = env
    grads = [torch.full((1000,), value, device="cuda"), torch.full((77,), -value, device="cuda")]
    out = torch.empty(2, device="cuda")
    wg.forge_grad_norm(wg.ForgeTensorList(grads), out, max_norm=1.0)
    x = float(np.float32(value))
    ref = math.sqrt(1077) * x
    coef = min(1.0, 1.0 / (ref + 1e-6))
    got = [float(t) for t in out.double().cpu()]
    if ref > float(np.finfo(np.float32).max):
        assert got[0] == math.inf                      # beyond float32
    else:
        # half a step: relative for normal results, 2^-150 for denormal ones
        assert abs(got[0] - ref) <= max(ref * U * 1.001, 2.0 ** -150)
    assert abs(got[1] - coef) <= max(coef * U * 1.001, 2.0 ** -150)


def test_norm_of_nonfinite_gradients(env):
    torch, wg = env
    for bad, norm, coef in ((math.inf, math.inf, 0.0), (math.nan, math.nan, math.nan)):
        for at in (0, 4097, 9999):
            g = torch.ones(10000, device="cuda")
            g[at] = bad
            out = torch.empty(2, device="cuda")
            wg.forge_grad_norm(wg.ForgeTensorList([torch.ones(3, device="cuda"), g]), out,
                               max_norm=1.0)
            got = out.cpu().numpy()
            np.testing.assert_array_equal(got, np.array([norm, coef], np.float32))


def test_norm_repeats_bitwise_and_counts_recurring_entries(env):
    torch, wg = env
    grads, *_ = make(torch, LISTS["many"], "both", 5)
    outs = [torch.empty(2, device="cuda") for _ in range(3)]
    for o in outs[:2]:
        wg.forge_grad_norm(wg.ForgeTensorList(grads), o, max_norm=1.0)
    assert torch.equal(outs[0], outs[1])
    wg.forge_grad_norm(wg.ForgeTensorList(grads + grads), outs[2], max_norm=1.0)
    ref = norm64(grads) * math.sqrt(2)
    check_norm(outs[2], ref, 1.0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", ["one", "odd", "chunk edges", "many", "large"])
def test_clip_grads(env, name, in_place):
    torch, wg = env
    grads, *_ = make(torch, LISTS[name], "both", 21)
    norm = torch.tensor([0.0, 0.37], device="cuda")
    want = [(g.float().cpu() * norm[1].cpu()).to(g.dtype) for g in grads]
    out = grads if in_place else [torch.full_like(g, 9.0) for g in grads]
    keep = [g.clone() for g in grads]
    wg.forge_clip_grads(wg.ForgeTensorList(grads, out=out), norm)
    for k, (o, w) in enumerate(zip(out, want)):
        assert torch.equal(o.cpu(), w), k
        assert in_place or torch.equal(grads[k], keep[k])


def adamw64(g, W, m, v, step, lr, beta1, beta2, eps, weight_decay):
    m1, v1 = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    den = (v1 / (1 - beta2 ** step)).sqrt() + eps
    s = lr / (1 - beta1 ** step)
    # Per element: two or three roundings and a rounded constant each of m and v; of the update,
    # besides what m and v pass on (half of v's), the square root, the reciprocal (1 ulp each), two
    # roundings of the denominator, two products and two constants.
    tm = 4 * U * (abs(beta1 * m) + abs((1 - beta1) * g))
    tv = 6 * U * v1
    tw = 4 * U * abs(W) + s / den * (tm + 16 * U * abs(m1))
    return (W * (1 - lr * weight_decay) - s * m1 / den, m1, v1), (tw, tm, tv)


def sgdm64(g, W, b, lr, momentum, weight_decay):
    b1 = momentum * b + g + weight_decay * W
    tb = 4 * U * (abs(momentum * b) + abs(g) + abs(weight_decay * W))
    return (W - lr * b1, b1), (4 * U * (abs(W) + abs(lr * b1)) + lr * tb, tb)


@pytest.mark.parametrize("dtypes", ["f32", "bf16", "both"])
@pytest.mark.parametrize("name", ["one", "odd", "chunk edges", "many", "large"])
def test_clipped_steps(env, name, dtypes):
    torch, wg = env
    grads, W, m, v = make(torch, LISTS[name], dtypes, 31)
    norm = torch.tensor([0.0, 0.61], device="cuda")
    g64 = [(g.float() * norm[1]).double().cpu() for g in grads]     # one float32 rounding
    st = [[t.clone() for t in ts] for ts in (W, m, v)]
    wg.forge_adamw_clipped(wg.ForgeTensorList(grads, W=st[0], m=st[1], v=st[2]), norm, **ADAM)
    for k in range(len(grads)):
        want, tol = adamw64(g64[k], *(ts[k].double().cpu() for ts in (W, m, v)), **ADAM)
        for got, w, t in zip(st, want, tol):
            assert bool(((got[k].double().cpu() - w).abs() <= t).all()), (k, LISTS[name][k])
    st = [[t.clone() for t in ts] for ts in (W, m)]
    wg.forge_sgdm_clipped(wg.ForgeTensorList(grads, W=st[0], mom=st[1]), norm, **SGDM)
    for k in range(len(grads)):
        want, tol = sgdm64(g64[k], *(ts[k].double().cpu() for ts in (W, m)), **SGDM)
        for got, w, t in zip(st, want, tol):
            assert bool(((got[k].double().cpu() - w).abs() <= t).all()), (k, LISTS[name][k])


@pytest.mark.parametrize("count", [63, 64, 65, 127, 128, 129, 160, 161, 257, 320, 321, 645])
def test_lists_of_any_length(env, count):
    # However the list is cut into launches, each tensor gets what it gets alone.
    torch, wg = env
    sizes = [1 + (k * 7919) % 6011 for k in range(count)]
    grads, W, m, v = make(torch, sizes, "both", 41)
    norm = torch.empty(2, device="cuda")
    wg.forge_grad_norm(wg.ForgeTensorList(grads), norm, max_norm=0.5)
    check_norm(norm, norm64(grads), 0.5)
    st, one = ([[t.clone() for t in ts] for ts in (W, m, v)] for _ in range(2))
    out, alone = [torch.full_like(g, 9.0) for g in grads], [torch.full_like(g, 9.0) for g in grads]
    wg.forge_adamw_clipped(wg.ForgeTensorList(grads, W=st[0], m=st[1], v=st[2]), norm, **ADAM)
    wg.forge_sgdm_clipped(wg.ForgeTensorList(grads, W=st[0], mom=st[1]), norm, **SGDM)
    wg.forge_clip_grads(wg.ForgeTensorList(grads, out=out), norm)
    for k in range(count):
        tensors = wg.ForgeTensorList(grads[k:k + 1], out=alone[k:k + 1], W=one[0][k:k + 1],
                                     m=one[1][k:k + 1], v=one[2][k:k + 1])
        wg.forge_adamw_clipped(tensors, norm, **ADAM)
        wg.forge_sgdm_clipped(tensors, norm, **SGDM)
        wg.forge_clip_grads(tensors, norm)
    torch.cuda.synchronize()
    for k in range(count):
        assert torch.equal(out[k], alone[k]), k
        assert all(torch.equal(a[k], b[k]) for a, b in zip(st, one)), k


@pytest.mark.parametrize("eps", [1e-8, 0.0])
def test_coefficient_one_is_the_unclipped_step(env, eps):
    torch, wg = env
    grads, W, m, v = make(torch, LISTS["odd"], "both", 41)
    norm = torch.tensor([0.0, 1.0], device="cuda")
    st, ref = ([[t.clone() for t in ts] for ts in (W, m, v)] for _ in range(2))
    hp = dict(ADAM, eps=eps)
    wg.forge_adamw_clipped(wg.ForgeTensorList(grads, W=st[0], m=st[1], v=st[2]), norm, **hp)
    for g, w, a, b in zip(grads, *ref):
        wg.forge_adamw_mixed(g, w, a, b, **hp)
    assert all(torch.equal(x, y) for xs, ys in zip(st, ref) for x, y in zip(xs, ys))
    st, ref = ([[t.clone() for t in ts] for ts in (W, m)] for _ in range(2))
    wg.forge_sgdm_clipped(wg.ForgeTensorList(grads, W=st[0], mom=st[1]), norm, **SGDM)
    for g, w, a in zip(grads, *ref):
        wg.forge_sgdm(g.float(), w, a, **SGDM)
    assert all(torch.equal(x, y) for xs, ys in zip(st, ref) for x, y in zip(xs, ys))


def test_neighbours_of_a_tensor_stay(env):
    torch, wg = env
    flat = [torch.full((64,), 3.0, device="cuda") for _ in range(4)]
    part = [f[16:16 + 21] for f in flat]                # 21 elements, 16-byte aligned, inside
    norm = torch.tensor([0.0, 0.5], device="cuda")
    wg.forge_adamw_clipped(wg.ForgeTensorList([part[0]], W=[part[1]], m=[part[2]], v=[part[3]]),
                           norm, **ADAM)
    wg.forge_clip_grads(wg.ForgeTensorList([part[0]], out=[part[0]]), norm)
    for f in flat:
        assert bool((f[:16] == 3).all()) and bool((f[37:] == 3).all())
        assert bool((f[16:37] != 3).all())


def test_graph_and_streams(env):
    torch, wg = env
    grads, W, m, v = make(torch, [5, 40000, 777], "both", 51)
    lists = wg.ForgeTensorList(grads, W=W, m=m, v=v)
    norm = torch.empty(2, device="cuda")
    ref = [[t.clone() for t in ts] for ts in (W, m, v)]
    ref_list = wg.ForgeTensorList(grads, W=ref[0], m=ref[1], v=ref[2])

    def step(ls):
        wg.forge_grad_norm(ls, norm, max_norm=0.5)
        wg.forge_adamw_clipped(ls, norm, **ADAM)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(lists)
    for k in range(4):                                  # new gradients in the same places
        for g in grads:
            g.mul_(1.5 if k % 2 else 0.5)
        graph.replay()
        torch.cuda.synchronize()
        step(ref_list)
        torch.cuda.synchronize()
        for xs, ys in zip((W, m, v), ref):
            assert all(torch.equal(x, y) for x, y in zip(xs, ys)), k
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty(2, device="cuda")
    torch.cuda.synchronize()
    wg.forge_grad_norm(lists, other, max_norm=0.5, stream=side)
    wg.forge_grad_norm(lists, norm, max_norm=0.5)       # beside it, its own workspace
    torch.cuda.synchronize()
    assert torch.equal(other, norm)


def test_binding_refuses(env):
    torch, wg = env
    g = torch.ones(8, device="cuda")
    norm = torch.ones(2, device="cuda")
    with pytest.raises(ValueError, match="without out"):
        wg.forge_clip_grads(wg.ForgeTensorList([g]), norm)
    with pytest.raises(ValueError, match="without v"):
        wg.forge_adamw_clipped(wg.ForgeTensorList([g], W=[g], m=[g]), norm, step=1)
    with pytest.raises(ValueError, match="contiguous"):
        wg.ForgeTensorList([torch.ones(8, 8, device="cuda").t()])
    with pytest.raises(wg.ForgeError, match="ALIAS"):
        wg.forge_sgdm_clipped(wg.ForgeTensorList([g], W=[g], mom=[g.clone()]), norm)
    with pytest.raises(wg.ForgeError, match="ALIGN"):
        wg.forge_grad_norm(wg.ForgeTensorList([g[1:]]), norm, max_norm=1.0)
    with pytest.raises(wg.ForgeError, match="HPARAM"):
        wg.forge_grad_norm(wg.ForgeTensorList([g]), norm, max_norm=-1.0)
    with pytest.raises(TypeError, match="ForgeTensorList"):
        wg.forge_grad_norm([g], norm, max_norm=1.0)
    with pytest.raises(ValueError, match="2 elements"):
        wg.forge_grad_norm(wg.ForgeTensorList([g]), g, max_norm=1.0)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(wg.ForgeError, match="SHAPE"):
        wg.forge_grad_norm(wg.ForgeTensorList([g]), norm, max_norm=1.0, workspace=small)
    assert bool((g == 1).all()) and bool((norm == 1).all())


def test_moved_tensors_are_refused_before_anything_runs(env):
    torch, wg = env
    sizes = [5000, 0, 77, 1]

    def data(t):
        t.data = t.clone()

    def grown(t):
        t.untyped_storage().resize_(4 * t.untyped_storage().nbytes() + (4 << 20))

    for move in (data, grown):
        for k in (0, 2, 3):
            for name, calls in (("grads", "nsac"), ("out", "c"), ("W", "sa"), ("m", "sa"), ("v", "a")):
                grads, W, m, v = make(torch, sizes, "f32", 7)
                fields = dict(grads=grads, out=[torch.ones_like(g) for g in grads], W=W, m=m, v=v)
                tensors = wg.ForgeTensorList(**fields)
                norm = torch.ones(2, device="cuda")
                move(fields[name][k])
                keep = {n: [t.clone() for t in ts] for n, ts in fields.items()}
                run = dict(n=lambda: wg.forge_grad_norm(tensors, norm, max_norm=1.0),
                           c=lambda: wg.forge_clip_grads(tensors, norm),
                           s=lambda: wg.forge_sgdm_clipped(tensors, norm, **SGDM),
                           a=lambda: wg.forge_adamw_clipped(tensors, norm, **ADAM))
                for call in calls:
                    with pytest.raises(ValueError, match=r"\[%d\] of the list is not where" % k):
                        run[call]()
                assert bool((norm == 1).all())
                for n, ts in fields.items():
                    assert all(torch.equal(a, b) for a, b in zip(ts, keep[n])), n


def test_list_over_a_training_loop(env):
    """A list built from the parameters' own gradients, over steps that clear
    them in place; gradients that backward made anew are refused."""
    torch, wg = env
    g = torch.Generator(device="cuda").manual_seed(3)
    layer = torch.nn.Linear(40, 24, device="cuda")
    W = list(layer.parameters())
    m, v = ([torch.zeros_like(w) for w in W] for _ in range(2))
    norm = torch.empty(2, device="cuda")

    def backward():
        x = torch.randn(9, 40, generator=g, device="cuda")
        layer(x).square().mean().backward()

    backward()
    tensors = wg.ForgeTensorList([w.grad for w in W], W=W, m=m, v=v)
    for step in range(1, 4):
        if step > 1:
            layer.zero_grad(set_to_none=False)
            backward()
        old = [[t.detach().double().cpu() for t in ts] for ts in (W, m, v)]
        wg.forge_grad_norm(tensors, norm, max_norm=0.01)
        wg.forge_adamw_clipped(tensors, norm, **dict(ADAM, step=step))
        check_norm(norm, norm64([w.grad for w in W]), 0.01)
        for k, w in enumerate(W):
            g64 = (w.grad * norm[1]).double().cpu()
            want, tol = adamw64(g64, *(ts[k] for ts in old), **dict(ADAM, step=step))
            for got, x, t in zip((w, m[k], v[k]), want, tol):
                assert bool(((got.detach().double().cpu() - x).abs() <= t).all()), (step, k)
    layer.zero_grad()
    backward()
    keep = [w.detach().clone() for w in W]
    for call in (lambda: wg.forge_grad_norm(tensors, norm, max_norm=0.01),
                 lambda: wg.forge_adamw_clipped(tensors, norm, **ADAM)):
        with pytest.raises(ValueError, match="another gradient"):
            call()
    assert all(torch.equal(a, b) for a, b in zip(W, keep))
