"""Layer norm, 8-bit products, distillation, embedding and clipped steps together, as
a distilling training step uses them: tokens -> lookup -> layer norm -> logits by an
8-bit product -> loss and gradient of the logits in place -> gradients of the
output layer, of the norm and of the embedding -> global norm -> clipped AdamW.
Each link is judged on what the link before it gave, in 64 bits; the whole step
captured in a graph gives the eager bits."""
import math

import pytest

from test_gpu_clip import adamw64
from test_gpu_distill import reference
from test_gpu_embedding import grad64, make_ids
from test_gpu_fp8_block import check_product, same
from test_gpu_layernorm import backward64, forward64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
T, V, D, OUT, VOCAB, K = 300, 211, 136, 264, 259, 7
TAU = 2.0


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


class Model:
    """Parameters, state and buffers: an embedding, a norm, and an output layer of 259
    words in 264 rows."""

    def __init__(self, torch, wg, seed):
        self.torch, self.wg = torch, wg
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.params = [torch.randn(V, D, generator=g, device="cuda") * 0.5,
                       1 + 0.1 * torch.randn(D, generator=g, device="cuda"),
                       0.1 * torch.randn(D, generator=g, device="cuda"),
                       torch.randn(OUT, D, generator=g, device="cuda") * 0.3]
        self.m = [torch.zeros_like(p) for p in self.params]
        self.v = [torch.zeros_like(p) for p in self.params]
        # The output layer's gradient is a product's: bf16.
        self.grads = [torch.empty_like(p) for p in self.params[:3]]
        self.grads.append(torch.empty(OUT, D, dtype=torch.bfloat16, device="cuda"))
        self.list = wg.ForgeTensorList(self.grads, W=self.params, m=self.m, v=self.v)
        self.norm, self.loss = torch.empty(2, device="cuda"), torch.empty(T, device="cuda")
        self.mean, self.rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        bf = dict(device="cuda", dtype=torch.bfloat16)
        self.X, self.Y, self.dY = (torch.empty(T, D, **bf) for _ in range(3))
        self.dX = torch.empty(T, D, **bf)
        self.logits = torch.empty(T, OUT, **bf)
        empty = wg.forge_fp8_block_empty
        self.q = {n: (empty(r, k, f), empty(k, r, f)) for n, r, k, f in
                  (("Y", T, D, "e4m3"), ("W", OUT, D, "e4m3"), ("dZ", T, OUT, "e5m2"))}
        self.seen = None

    def quantize(self, name, x, **kw):
        rows, cols = self.q[name]
        self.wg.forge_quantize_fp8_block(x, rows=rows, cols=cols, **kw)
        return rows, cols

    def step(self, ids, teacher, words, weight, step, watch=False):
        wg, (emb, gamma, beta, W) = self.wg, self.params
        wg.forge_embedding(emb, ids, self.X, scale=math.sqrt(D))
        wg.forge_layernorm(self.X, gamma, beta, self.Y, self.mean, self.rstd)
        yr, yc = self.quantize("Y", self.Y)
        wr, wc = self.quantize("W", W, square=True)
        wg.forge_matmul_fp8_block(yr, wr, self.logits)
        if watch:
            self.seen = self.logits.clone()
        wg.forge_distill(self.logits, teacher, words, self.loss, self.logits, vocab=VOCAB,
                         weight=weight, temperature=TAU, scale=1.0 / T)
        zr, zc = self.quantize("dZ", self.logits)
        wg.forge_matmul_fp8_block(zr, wc, self.dY)
        wg.forge_matmul_fp8_block(zc, yc, self.grads[3])
        wg.forge_layernorm_backward(self.dY, self.X, gamma, self.mean, self.rstd, self.dX,
                                    self.grads[1], self.grads[2])
        wg.forge_embedding_grad(ids, self.dX, self.grads[0], scale=math.sqrt(D))
        wg.forge_grad_norm(self.list, self.norm, max_norm=0.01)
        wg.forge_adamw_clipped(self.list, self.norm, step=step, **HP)

    def state(self):
        return [t.clone() for t in (*self.params, *self.m, *self.v, self.norm, self.loss, self.dX)]


def batch(torch, seed):
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    ids = make_ids(torch, T, V, "zipf", torch.int64, seed=seed).cuda()
    teacher = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    words = torch.randint(-1, VOCAB, (T, K), generator=g, device="cuda")
    weight = (torch.rand(T, generator=g, device="cuda") > 0.1).float()
    return ids, teacher, words, weight


def within(got, want, tol, what):
    assert bool(((got.double() - want).abs() <= tol).all()), what


def test_step_link_by_link(env):
    torch, wg = env
    M = Model(torch, wg, 1)
    for t in (1, 2, 3):
        ids, teacher, words, weight = batch(torch, t)
        old = [[x.clone() for x in xs] for xs in (M.params, M.m, M.v)]
        M.step(ids, teacher, words, weight, t, watch=True)
        _, gamma, beta, W = old[0]
        want = forward64(torch, M.X, gamma, beta, 1e-5, "bfloat16")
        within(M.Y, want[0], want[3], "Y")
        within(M.mean, want[1], want[4], "mean")
        within(M.rstd, want[2], want[5], "rstd")
        for name, x, square in (("Y", M.Y, False), ("W", W, True), ("dZ", M.logits, False)):
            same(torch, M.q[name][0], x, square)
            same(torch, M.q[name][1], x.t(), square)
        check_product(torch, M.seen, M.q["Y"][0], M.q["W"][0])
        want = reference(torch, M.seen, teacher, words, weight, VOCAB, TAU, 1.0 / T, "bfloat16")
        within(M.loss, want[0], want[2], "loss")
        within(M.logits, want[1], want[3], "gradient of the logits")
        assert not M.logits[:, VOCAB:].any()
        check_product(torch, M.dY, M.q["dZ"][0], M.q["W"][1])
        check_product(torch, M.grads[3], M.q["dZ"][1], M.q["Y"][1])
        want = backward64(torch, M.dY, M.X, gamma, M.mean, M.rstd, "bfloat16")
        for k, got in enumerate((M.dX, M.grads[1], M.grads[2])):
            within(got, want[k], want[3 + k], ("dX", "dgamma", "dbeta")[k])
        want, tol, _ = grad64(torch, ids, M.dX, V, math.sqrt(D))
        assert bool(((M.grads[0].double().cpu() - want).abs() <= tol).all())
        norm = math.sqrt(sum(float((g.double() ** 2).sum()) for g in M.grads))
        assert abs(float(M.norm[0]) - norm) <= norm * U * 1.001
        for k in range(4):
            g = (M.grads[k].float() * M.norm[1]).double().cpu()
            want, tol = adamw64(g, *(xs[k].double().cpu() for xs in old), t, **HP)
            for got, w, tl in zip((M.params[k], M.m[k], M.v[k]), want, tol):
                assert bool(((got.double().cpu() - w).abs() <= tl).all()), (t, k)


def test_captured_step_gives_the_eager_bits(env):
    torch, wg = env
    A, B = Model(torch, wg, 2), Model(torch, wg, 2)
    fixed = batch(torch, 0)
    A.step(*fixed, 1)
    B.step(*fixed, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.step(*fixed, 2)
    for k in range(4):
        for into, x in zip(fixed, batch(torch, 10 + k)):
            into.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        B.step(*fixed, 2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(A.state(), B.state())), k


def test_two_models_side_by_side(env):
    """Two captured steps, each with the workspaces of its capture, replayed on two streams at
    once."""
    torch, wg = env
    data = batch(torch, 3)
    models, alone = ([Model(torch, wg, s) for s in (5, 6)] for _ in range(2))
    graphs = []
    torch.cuda.synchronize()
    for M in models:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            M.step(*data, 1)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for M, R in zip(models, alone):
        for _ in range(3):
            R.step(*data, 1)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(M.state(), R.state()))


def test_the_gradient_of_the_logits_feeds_the_fused_step(env):
    """dY of the LM head as it is: the bf16 gradient, written over the logits, into the weight
    gradient with the optimizer behind it."""
    torch, wg = env
    g = torch.Generator(device="cuda").manual_seed(4)
    X = torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn(OUT, D, generator=g, device="cuda") * 0.3
    logits = torch.randn(T, OUT, generator=g, device="cuda").to(torch.bfloat16)
    _, teacher, words, weight = batch(torch, 9)
    loss = torch.empty(T, device="cuda")
    wg.forge_distill(logits, teacher, words, loss, logits, vocab=VOCAB, weight=weight, scale=1.0 / T)
    m, v, grad = torch.zeros_like(W), torch.zeros_like(W), torch.empty_like(W)
    wg.forge_wgrad(X, logits, grad)
    assert not grad[VOCAB:].any() and grad[:VOCAB].any()
    want = logits.double().t() @ X.double()
    size = logits.double().abs().t() @ X.double().abs()
    assert bool(((grad.double() - want).abs() <= (T / 16 + 16) * U * size).all())
    W2, m2, v2 = W.clone(), m.clone(), v.clone()
    wg.forge_wgrad_adamw(X, logits, W, m, v, step=1, weight_decay=0.0)
    wg.forge_adamw(grad, W2, m2, v2, step=1, weight_decay=0.0)
    assert torch.equal(W, W2) and torch.equal(m, m2) and torch.equal(v, v2)
