"""Timing cases of three more operators of a training step.

Each in plain torch (`own` false) and as the library's calls (`own` true):

  layer norm    forward, and backward with the reduction of the weight's and
                the bias's gradients over the tokens
  fp8 block     8-bit floating point operands with a power-of-two scale for
                each block of 128 values, and their product: a layer's output,
                its input gradient and its weight gradient
  distillation  the loss of a student's logits against a teacher's top logits
                at a temperature, and its gradient

Sizes are those of the repository's own workloads (MLP-down 14336 -> 4096,
QKV 4096 -> 6144, LM head 4096 -> 128256) or generic.
"""
import math

import torch

own = False

VOCAB, WIDTH = 128256, 4096
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}
SIZE = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
EPS = 1e-5
#: Mantissa bits, least normal exponent and largest value of the 8-bit formats.
FORMAT = {"e4m3": (3, -6, 448.0, torch.float8_e4m3fn), "e5m2": (2, -14, 57344.0, torch.float8_e5m2)}


def listed():
    return [
        # The norm before a projection for one decoded token: latency alone.
        {"name": "layer norm 1 token", "op": "lnfwd", "T": 1, "d": WIDTH, "x": "f32", "y": "bf16"},
        # The norm of a training batch in bf16.
        {"name": "layer norm 16384 tokens", "op": "lnfwd", "T": 16384, "d": WIDTH, "x": "bf16", "y": "bf16"},
        # A narrow model's backward in float32, an odd batch.
        {"name": "layer norm backward small", "op": "lnbwd", "T": 333, "d": 1000, "x": "f32", "y": "f32"},
        # The backward of a training batch, residual stream and gradients in bf16.
        {"name": "layer norm backward 16384", "op": "lnbwd", "T": 16384, "d": WIDTH, "x": "bf16", "y": "bf16"},
        # One decoded token through MLP-down, its weight held in 8 bits.
        {"name": "fp8 output 1 token", "op": "fp8fwd", "T": 1, "d_in": 14336, "d_out": 4096, "x": "bf16", "w": "kept", "dy": "e4m3"},
        # A small layer's output, an odd number of tokens, activations in float32.
        {"name": "fp8 output small", "op": "fp8fwd", "T": 333, "d_in": 1024, "d_out": 520, "x": "f32", "w": "kept", "dy": "e4m3"},
        # MLP-down's output in training: the float32 master weight quantised anew, as it changes every step.
        {"name": "fp8 output mlp-down", "op": "fp8fwd", "T": 8192, "d_in": 14336, "d_out": 4096, "x": "bf16", "w": "fresh", "dy": "e4m3"},
        # QKV's weight gradient: both operands quantised along the tokens.
        {"name": "fp8 weight gradient qkv", "op": "fp8wgrad", "T": 16384, "d_in": 4096, "d_out": 6144, "x": "bf16", "w": "kept", "dy": "e5m2"},
        # The loss alone, as in an evaluation, float32 logits of an odd vocabulary.
        {"name": "distillation loss", "op": "loss", "T": 511, "V": 50021, "K": 64, "z": "f32", "g": "f32", "u": "f32", "ids": "i64", "tau": 1.0},
        # A few positions of a large vocabulary.
        {"name": "distillation 8 rows", "op": "distill", "T": 8, "V": VOCAB, "K": 20, "z": "bf16", "g": "bf16", "u": "bf16", "ids": "i32", "tau": 2.0},
        # A mid-sized model: float32 logits, the gradient in bf16 for the weight gradient behind it.
        {"name": "distillation 1021 rows", "op": "distill", "T": 1021, "V": 32003, "K": 128, "z": "f32", "g": "bf16", "u": "f32", "ids": "i32", "tau": 1.5},
        # The LM head's batch.
        {"name": "distillation lm head", "op": "distill", "T": 4096, "V": VOCAB, "K": 64, "z": "bf16", "g": "bf16", "u": "bf16", "ids": "i64", "tau": 2.0},
    ]


def draw(rng):
    def logint(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    def mult8(a, b):
        return 8 * logint(a // 8, b // 8)

    op = rng.choice(["lnfwd", "lnbwd", "fp8fwd", "fp8dgrad", "fp8wgrad", "loss", "distill"])
    while True:
        if op in ("lnfwd", "lnbwd"):
            c = {"op": op, "T": logint(1, 65536), "d": mult8(64, 16384), "x": rng.choice(["f32", "bf16"]), "y": rng.choice(["f32", "bf16"])}
            if c["T"] * c["d"] <= 16384 * WIDTH:
                return c
        elif op in ("loss", "distill"):
            c = {"op": op, "T": logint(1, 16384), "V": logint(1000, VOCAB), "K": logint(1, 256), "z": rng.choice(["f32", "bf16"]),
                 "g": rng.choice(["f32", "bf16"]), "u": rng.choice(["f32", "bf16"]), "ids": rng.choice(["i32", "i64"]),
                 "tau": rng.choice([1.0, 1.5, 2.0, 4.0])}
            if c["T"] * c["V"] <= 2048 * VOCAB:
                return c
        else:
            c = {"op": op, "T": logint(1, 16384), "d_in": mult8(64, 14336), "d_out": mult8(64, 14336), "x": rng.choice(["f32", "bf16"]),
                 "w": rng.choice(["kept", "fresh"]), "dy": rng.choice(["e4m3", "e5m2"])}
            if c["T"] * c["d_in"] * c["d_out"] <= 8192 * 14336 * 4096 and c["d_in"] * c["d_out"] <= 14336 * 6144:
                return c


def _pitch(V):
    """Columns of a row of logits in memory: the vocabulary padded to whole vectors."""
    return (V + 7) // 8 * 8


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}

    def normal(shape, dtype="f32", std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(DTYPE[dtype])

    if op in ("lnfwd", "lnbwd"):
        T, d = case["T"], case["d"]
        # A residual stream: every channel with its own mean and width, some of them large.
        width = torch.exp(normal((d,), std=0.7))
        x = normal((T, d)).mul_(width).add_(normal((d,), std=0.3))
        s["x"] = x.to(DTYPE[case["x"]])
        s["gamma"] = normal((d,), std=0.1).add_(1.0)
        if op == "lnfwd":
            s["beta"] = normal((d,), std=0.1)
            s["y"] = torch.empty((T, d), dtype=DTYPE[case["y"]], device="cuda")
            s["mean"], s["rstd"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        else:
            s["dY"] = normal((T, d), case["y"], 1e-2)
            v, m = torch.var_mean(s["x"].double() if T * d < 1 << 24 else s["x"].float(), 1, correction=0)
            s["mean"], s["rstd"] = m.float(), (v + EPS).rsqrt().float()
            s["dX"] = torch.empty_like(s["x"])
            s["dgamma"], s["dbeta"] = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    elif op in ("loss", "distill"):
        T, V, K = case["T"], case["V"], case["K"]
        # Teacher: the largest logits in falling order, one entry in 16 unused (-1), as for rows with fewer of them.
        u = torch.sort(normal((T, K), std=2.0).add_(12.0), descending=True).values
        s["teacher"] = u.to(DTYPE[case["u"]])
        ids = torch.randint(0, V, (T, K), generator=g, device="cuda")
        hidden = torch.rand((T, K), generator=g, device="cuda") < 1 / 16
        s["ids"] = torch.where(hidden, -1, ids).to(DTYPE[case["ids"]])
        # Student: it knows the teacher's tokens in part.
        z = normal((T, _pitch(V)), std=2.0)
        z.scatter_reduce_(1, ids, u * 0.8 + normal((T, K)), "amax")
        z[:, V:] = 1e4                                      # what a padded output layer leaves there
        s["logits"] = z.to(DTYPE[case["z"]])
        # One row in 8 is padding.
        s["weight"] = (torch.rand(T, generator=g, device="cuda") >= 1 / 8).float()
        s["scale"] = 1.0 / T
        s["loss"] = torch.empty(T, device="cuda")
        if op == "distill":
            s["grad"] = torch.empty((T, _pitch(V)), dtype=DTYPE[case["g"]], device="cuda")
    else:
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        if op != "fp8dgrad":
            # Activations with channels of different size.
            s["X"] = normal((T, d_in)).mul_(torch.exp(normal((d_in,), std=0.7))).to(DTYPE[case["x"]])
        if op != "fp8fwd":
            s["dY"] = normal((T, d_out), case["x"], 1e-2)
        if op != "fp8wgrad":
            s["W"] = normal((d_out, d_in), std=0.02)
        shape = {"fp8fwd": (T, d_out), "fp8dgrad": (T, d_in), "fp8wgrad": (d_out, d_in)}[op]
        s["out"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        if op != "fp8wgrad" and case["w"] == "kept":      # a weight that is laid out once
            if own:
                import weight_gradient_gemm_amd as wg
                rows = op == "fp8fwd"
                s["W8"] = wg.forge_fp8_block_empty(d_out, d_in) if rows else wg.forge_fp8_block_empty(d_in, d_out)
                wg.forge_quantize_fp8_block(s["W"], square=True, **{"rows" if rows else "cols": s["W8"]})
            else:
                s["W8"] = _fp8_block(s["W"], "e4m3", True)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _fp8_block(x, fmt, square=False):
    """The values that x [R, K] stands for in 8 bits: blocks of 128 along K (and of 128 rows where
    `square`) share the least power of two that brings them into the format's range."""
    _, _, top, dtype = FORMAT[fmt]
    R, K = x.shape
    rows, cols = (R + 127) // 128, (K + 127) // 128
    b = torch.zeros((rows * 128, cols * 128), device=x.device)
    b[:R, :K] = x
    b = b.view(rows, 128, cols, 128)
    amax = b.abs().amax((1, 3) if square else 3, keepdim=True)
    # The biased exponent, one more where the fraction lies beyond the largest code's, less the format's reach.
    carry = (1 << 23) - 1 - (int(math.frexp(top)[0] * 2 ** 24) - 2 ** 23)
    e = ((amax.view(torch.int32) + carry) >> 23) - (math.frexp(top)[1] - 1)
    e = e.clamp(min=0)
    up, down = ((254 - e) << 23).view(torch.float32), (e.clamp(min=1) << 23).view(torch.float32)
    q = (b * up).to(dtype).float() * torch.where(e > 0, down, 2.0 ** -127)
    return q.view(rows * 128, cols * 128)[:R, :K]


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "lnfwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = ((x * x).mean(1, keepdim=True) + EPS).rsqrt()
        s["y"].copy_(x * rstd * s["gamma"] + s["beta"])
        return s["y"], mean[:, 0], rstd[:, 0]
    if op == "lnbwd":
        dy = s["dY"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        a = dy * s["gamma"]
        dx = s["rstd"][:, None] * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
        s["dX"].copy_(dx)
        return s["dX"], (dy * xhat).sum(0), dy.sum(0)
    if op in ("loss", "distill"):
        V, tau = case["V"], case["tau"]
        z = s["logits"][:, :V].float() / tau
        m = z.amax(1, keepdim=True)
        p = torch.exp(z - m)
        total = p.sum(1, keepdim=True)
        ids = s["ids"].long()
        kept = ids >= 0
        at = ids.clamp(min=0)
        u = torch.where(kept, s["teacher"].float() / tau, -math.inf)
        some = kept.any(1, keepdim=True)
        u = torch.where(some, u, 0.0)
        e = torch.exp(u - u.amax(1, keepdim=True))
        q = torch.where(kept, e / e.sum(1, keepdim=True), 0.0)
        logp = z.gather(1, at) - m - total.log()
        w = s["scale"] * s["weight"][:, None] * some
        terms = torch.where(q > 0, q * (q.clamp(min=1e-38).log() - logp), 0.0)
        loss = (w * tau * tau * terms.sum(1, keepdim=True))[:, 0]
        if op == "loss":
            return loss
        grad = (p / total).scatter_add_(1, at, -q) * (w * tau)
        s["grad"][:, :V] = grad
        s["grad"][:, V:] = 0
        return loss, s["grad"]
    dy = case["dy"]
    if op == "fp8wgrad":
        s["out"].copy_(_fp8_block(s["dY"].t(), dy) @ _fp8_block(s["X"].t(), "e4m3").t())
        return s["out"]
    W = s["W8"] if case["w"] == "kept" else _fp8_block(s["W"], "e4m3", True)
    if op == "fp8fwd":
        s["out"].copy_(_fp8_block(s["X"], "e4m3") @ W.t())
    else:
        s["out"].copy_(_fp8_block(s["dY"], dy) @ W)
    return s["out"]


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------
def _own(s):
    import weight_gradient_gemm_amd as wg
    case = s["case"]
    op = case["op"]
    if op == "lnfwd":
        wg.forge_layernorm(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return s["y"], s["mean"], s["rstd"]
    if op == "lnbwd":
        wg.forge_layernorm_backward(s["dY"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dX"], s["dgamma"], s["dbeta"])
        return s["dX"], s["dgamma"], s["dbeta"]
    if op in ("loss", "distill"):
        wg.forge_distill(s["logits"], s["teacher"], s["ids"], s["loss"], s.get("grad"), vocab=case["V"], weight=s["weight"],
                         temperature=case["tau"], scale=s["scale"])
        return s["loss"] if op == "loss" else (s["loss"], s["grad"])
    T, d_in, d_out, dy = case["T"], case["d_in"], case["d_out"], case["dy"]
    if op == "fp8wgrad":
        dY, X = wg.forge_fp8_block_empty(d_out, T, dy), wg.forge_fp8_block_empty(d_in, T)
        wg.forge_quantize_fp8_block(s["dY"], cols=dY)
        wg.forge_quantize_fp8_block(s["X"], cols=X)
        wg.forge_matmul_fp8_block(dY, X, s["out"])
        return s["out"]
    if op == "fp8fwd":
        W = s["W8"] if case["w"] == "kept" else wg.forge_fp8_block_empty(d_out, d_in)
        if case["w"] == "fresh":
            wg.forge_quantize_fp8_block(s["W"], rows=W, square=True)
        X = wg.forge_fp8_block_empty(T, d_in)
        wg.forge_quantize_fp8_block(s["X"], rows=X)
        wg.forge_matmul_fp8_block(X, W, s["out"])
        return s["out"]
    W = s["W8"] if case["w"] == "kept" else wg.forge_fp8_block_empty(d_in, d_out)
    if case["w"] == "fresh":
        wg.forge_quantize_fp8_block(s["W"], cols=W, square=True)
    dY = wg.forge_fp8_block_empty(T, d_out, dy)
    wg.forge_quantize_fp8_block(s["dY"], rows=dY)
    wg.forge_matmul_fp8_block(dY, W, s["out"])
    return s["out"]


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("lnfwd", "lnbwd"):
        n, x, y = case["T"] * case["d"], SIZE[case["x"]], SIZE[case["y"]]
        if op == "lnfwd":
            return {"bytes": n * (x + y) + 8 * case["T"] + 8 * case["d"], "flops": 8 * n}
        return {"bytes": n * (2 * x + y) + 8 * case["T"] + 12 * case["d"], "flops": 14 * n}
    if op in ("loss", "distill"):
        T, n = case["T"], case["T"] * case["V"]
        entries = T * case["K"] * (SIZE[case["u"]] + SIZE[case["ids"]]) + 8 * T
        if op == "loss":
            return {"bytes": n * SIZE[case["z"]] + entries, "flops": 4 * n}
        return {"bytes": n * (SIZE[case["z"]] + SIZE[case["g"]]) + entries, "flops": 8 * n}
    T, d_in, d_out, b = case["T"], case["d_in"], case["d_out"], SIZE[case["x"]]
    flops = 2 * T * d_in * d_out
    if op == "fp8wgrad":
        return {"bytes": T * (d_in + d_out) * b + 2 * d_in * d_out, "flops": flops}
    # A weight that is kept is a byte a value, a fresh one comes in float32.
    weight = d_in * d_out * (1 if case["w"] == "kept" else 4)
    k, n = (d_in, d_out) if op == "fp8fwd" else (d_out, d_in)
    return {"bytes": T * k * b + weight + 2 * T * n, "flops": flops}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def layer_norm(x):
        x = x.to(f64)
        mu = x.sum(1) / x.shape[1]
        var = (x - mu[:, None]).pow(2).sum(1) / x.shape[1]
        r = 1.0 / torch.sqrt(var + EPS)
        return (x - mu[:, None]) * r[:, None] * s["gamma"].to(f64) + s["beta"].to(f64), mu, r

    def layer_norm_backward():
        T, d = case["T"], case["d"]
        dx = torch.empty((T, d), dtype=f64, device="cuda")
        dg, db = torch.zeros(d, dtype=f64, device="cuda"), torch.zeros(d, dtype=f64, device="cuda")
        rows = max(1, (1 << 25) // d)
        for t in range(0, T, rows):
            part = slice(t, t + rows)
            dy, r = s["dY"][part].to(f64), s["rstd"][part].to(f64)[:, None]
            n = (s["x"][part].to(f64) - s["mean"][part].to(f64)[:, None]) * r
            dg += (dy * n).sum(0)
            db += dy.sum(0)
            dy = dy * s["gamma"].to(f64)
            dx[part] = r * (dy - (dy.sum(1, keepdim=True) + n * (dy * n).sum(1, keepdim=True)) / d)
        return dx, dg, db

    def distill():
        T, V, K, tau = case["T"], case["V"], case["K"], case["tau"]
        losses = torch.zeros(T, dtype=f64, device="cuda")
        grads = torch.zeros((T, _pitch(V)), dtype=f64, device="cuda") if op == "distill" else None
        rows = max(1, (1 << 25) // V)
        for t in range(0, T, rows):
            part = slice(t, t + rows)
            logp = torch.log_softmax(s["logits"][part, :V].to(f64) / tau, 1)
            ids = s["ids"][part].to(torch.int64)
            u = torch.where(ids < 0, torch.tensor(-math.inf, dtype=f64, device="cuda"), s["teacher"][part].to(f64) / tau)
            w = s["weight"][part].to(f64) * s["scale"] * (ids >= 0).any(1)
            logq = torch.where(w[:, None] > 0, torch.log_softmax(u, 1), -math.inf)
            q = torch.exp(logq)
            at = torch.where(ids < 0, 0, ids)
            diff = torch.where(q > 0, logq - torch.take_along_dim(logp, at, 1), 0.0)
            losses[part] = w * tau ** 2 * (q * diff).sum(1)
            if grads is not None:
                target = torch.zeros_like(logp).scatter_add_(1, at, q)
                grads[part, :V] = (torch.exp(logp) - target) * (w * tau)[:, None]
        return losses if grads is None else (losses, grads)

    def rounded(x, fmt, square=False):
        """Each block of 128 divided by its power of two, and each value rounded to the nearest multiple
        of the spacing that the format has there (halves to the even one)."""
        mantissa, lowest, top, _ = FORMAT[fmt]
        tf, te = math.frexp(top)
        out = torch.empty(x.shape, dtype=f64, device="cuda")
        for r in range(0, x.shape[0], 1024):
            for c in range(0, x.shape[1], 8192):
                part = x[r:r + 1024, c:c + 8192].to(f64)
                full = torch.nn.functional.pad(part, (0, -part.shape[1] % 128, 0, -part.shape[0] % 128))
                blocks = full.unflatten(1, (-1, 128)).unflatten(0, (-1, 128))       # [R / 128, 128, K / 128, 128]
                largest = blocks.abs().amax(3, keepdim=True)
                if square:
                    largest = largest.amax(1, keepdim=True)
                f, e = torch.frexp(largest)
                e = torch.where(largest > 0, e.to(torch.int64) - te + (f > tf), -127).clamp(min=-127)
                power = ((e + 1023) << 52).view(f64)
                y = blocks / power
                spacing = torch.frexp(y)[1].to(torch.int64).sub_(1).clamp_(min=lowest).sub_(mantissa)
                spacing = ((spacing + 1023) << 52).view(f64)
                y = torch.round(y / spacing) * spacing * power
                out[r:r + 1024, c:c + 8192] = y.flatten(2, 3).flatten(0, 1)[:part.shape[0], :part.shape[1]]
        return out

    if op == "lnfwd":
        return layer_norm(s["x"])
    if op == "lnbwd":
        return layer_norm_backward()
    if op in ("loss", "distill"):
        return distill()
    if op == "fp8wgrad":
        return torch.matmul(rounded(s["dY"].t(), case["dy"]), rounded(s["X"].t(), "e4m3").t())
    W = rounded(s["W"], "e4m3", True)
    if op == "fp8fwd":
        return torch.matmul(rounded(s["X"], "e4m3"), W.t())
    return torch.matmul(rounded(s["dY"], case["dy"]), W)
