"""Microscaled 4-bit quantisation and products on the GPU against their
definitions in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                  # half a float32 step, relative
ADAM = dict(step=5, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
TILES = (0, 1, 2, 3, 4)


@pytest.fixture(scope="module")
def env():
    import torch
    import weight_gradient_gemm_amd as wg
    return torch, wg


def reference(torch, x):
    """x [R, K] in blocks of 32 along K: values [R, Kp] float64 (NaN blocks
    included) and scale bytes [R, Kp / 32], by comparing against the borders."""
    R, K = x.shape
    Kp = (K + 127) // 128 * 128
    b = torch.zeros(R, Kp, dtype=torch.float64)
    b[:, :K] = x.double().cpu()
    b = b.view(R, Kp // 32, 32)
    bad = ~torch.isfinite(b).all(2)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top)[1].long() - 3, -127).clamp(min=-127)
    power = ((e + 1023) << 52).view(torch.float64)[..., None]
    y = b.abs() / power
    q = torch.zeros_like(y)
    for border, up, tie in ((0.25, 0.5, False), (0.75, 0.5, True), (1.25, 0.5, False),
                            (1.75, 0.5, True), (2.5, 1.0, False), (3.5, 1.0, True),
                            (5.0, 2.0, False)):
        q += up * ((y >= border) if tie else (y > border))
    q = q * torch.sign(b) * power
    q = torch.where(bad[..., None], torch.full_like(q, math.nan), q)
    return q.view(R, Kp), torch.where(bad, 255, e + 127)


def decode(torch, operand):
    """The values of an operand, and its scale bytes by row and block."""
    codes, scales = operand.codes.cpu(), operand.scales.cpu()
    codes = codes.permute(1, 0, 2).reshape(codes.shape[1], -1)
    R, half = codes.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    table = torch.cat([table, -table])
    v = table[torch.stack([codes & 15, codes >> 4], 2).long().view(R, 2 * half)]
    s = scales.permute(1, 0, 2).reshape(R, -1).long()
    p = torch.where(s == 255, torch.full(s.shape, math.nan, dtype=torch.float64),
                    ((s - 127 + 1023) << 52).view(torch.float64))
    return (v.view(R, -1, 32) * p[..., None]).view(R, 2 * half), s


def same(torch, operand, x):
    want, bytes_ = reference(torch, x)
    got, s = decode(torch, operand)
    assert torch.equal(s, bytes_)
    assert torch.equal(torch.nan_to_num(got, nan=1e300), torch.nan_to_num(want, nan=1e300))


def both(torch, wg, x):
    R, C = x.shape
    rows, cols = wg.forge_mxfp4_empty(R, C), wg.forge_mxfp4_empty(C, R)
    for op in (rows, cols):
        op.codes.fill_(0xA5)
        op.scales.fill_(0xA5)
    wg.forge_quantize_mxfp4(x, rows=rows, cols=cols)
    return rows, cols


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,C", [(1, 8), (1, 128), (33, 40), (128, 128), (129, 136), (31, 264),
                                 (333, 520), (1000, 1032), (257, 8)])
def test_quantize(env, R, C, dtype):
    torch, wg = env
    g = torch.Generator().manual_seed(R * C)
    x = (torch.randn(R, C, generator=g) * torch.exp(torch.randn(R, C, generator=g) * 3)).to(
        getattr(torch, dtype)).cuda()
    rows, cols = both(torch, wg, x)
    same(torch, rows, x)
    same(torch, cols, x.t())
    # each alone gives the same bytes
    one, two = wg.forge_mxfp4_empty(R, C), wg.forge_mxfp4_empty(C, R)
    wg.forge_quantize_mxfp4(x, rows=one)
    wg.forge_quantize_mxfp4(x, cols=two)
    for a, b in ((rows, one), (cols, two)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_borders_at_every_exponent(env, dtype):
    """Every multiple of 1/32 up to 8 (all borders and both sides of them),
    under each size of a block's largest, at exponents down to the denormals."""
    torch, wg = env
    grid = torch.arange(0, 256, dtype=torch.float64) / 32
    exps = [-149, -140, -130, -127, -126, -125, -100, -96, -95, -94, -93, -92, -64, -1, 0, 1, 63,
            100, 124]
    blocks = []
    for k in exps:
        for top in (4.0, 5.0, 6.0, 7.75):
            vals = grid[grid <= top]
            vals = torch.cat([vals, -vals])
            pad = -len(vals) % 31
            vals = torch.cat([vals, torch.zeros(pad, dtype=torch.float64)]).view(-1, 31)
            lead = torch.full((len(vals), 1), top, dtype=torch.float64)
            blocks.append(torch.cat([lead, vals], 1) * 2.0 ** k)
    x = torch.cat(blocks)
    x = torch.cat([x, torch.zeros(-len(x) % 4, 32, dtype=torch.float64)]).view(-1, 128)
    x = x.to(getattr(torch, dtype)).cuda()          # rounds what a denormal cannot hold
    rows, _ = both(torch, wg, x)
    same(torch, rows, x)
    xt = x.t().contiguous()
    xt = torch.nn.functional.pad(xt, (0, -xt.shape[1] % 8))
    _, cols = both(torch, wg, xt)
    same(torch, cols, xt.t())


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_nonfinite_blocks(env, dtype):
    torch, wg = env
    x = torch.randn(64, 256).to(getattr(torch, dtype))
    x[3, 40], x[7, 255], x[33, 0], x[63, 128] = math.nan, math.inf, -math.inf, math.nan
    x = x.cuda()
    rows, cols = both(torch, wg, x)
    same(torch, rows, x)
    same(torch, cols, x.t())


def operands(torch, wg, M, N, K, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def one(R):
        x = torch.randn(R, K, generator=g) * torch.exp(torch.randn(R, 1, generator=g) * spread)
        pad = torch.nn.functional.pad(x, (0, -K % 8)).cuda()
        op = wg.forge_mxfp4_empty(R, K)
        wg.forge_quantize_mxfp4(pad, rows=op)
        return op

    return one(M), one(N)


def product64(torch, A, B):
    a, b = decode(torch, A)[0], decode(torch, B)[0]
    return a @ b.t(), a.abs() @ b.abs().t(), a.shape[1]


def check_product(torch, out, A, B):
    want, size, K = product64(torch, A, B)
    # Products of codes are exact. Whatever the instruction's order, an element is the sum of K
    # of them in float32, each addition off by at most a whole step (if it truncates) of a partial
    # sum that the magnitudes bound; at most one addition in 8 products and one a step of 64.
    tol = (K / 8 + K / 64 + 2) * 2 * U * size
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


SHAPES = [(1, 8, 1), (1, 8, 128), (3, 16, 129), (128, 128, 256), (129, 136, 333), (255, 264, 512),
          (257, 520, 641), (520, 1024, 333), (1, 4096, 1000), (700, 8, 2048), (300, 1032, 5000)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(env, M, N, K, dtype):
    torch, wg = env
    A, B = operands(torch, wg, M, N, K, M + N + K)
    outs = []
    for tile in TILES:
        guard = torch.full((M * N + 64,), 7.0, dtype=getattr(torch, dtype), device="cuda")
        out = guard[:M * N].view(M, N)
        wg.forge_matmul_mxfp4(A, B, out, tile=tile)
        assert bool((guard[M * N:] == 7).all())
        outs.append(out)
    check_product(torch, outs[0], A, B)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_matmul_of_nan_in_the_last_rows(env):
    # The rows past a tile's edge repeat the last one.
    torch, wg = env
    A, B = operands(torch, wg, 70, 136, 700, 3)
    A.scales[2, 69, 1] = 255
    out = torch.empty(70, 136, device="cuda")
    for tile in TILES:
        wg.forge_matmul_mxfp4(A, B, out, tile=tile)
        assert bool(torch.isnan(out[69]).all()) and bool(torch.isfinite(out[:69]).all())


def test_matmul_of_an_operand_beyond_31_bits(env):
    # 2.7 GB of codes: rows of the large operand give what they give in a small one.
    torch, wg = env
    N, K, M = (1 << 21) + 8, 2560, 3
    g = torch.Generator(device="cuda").manual_seed(4)

    def random(R):
        codes = torch.randint(0, 256, (K // 128, R, 64), dtype=torch.uint8, device="cuda", generator=g)
        scales = torch.randint(120, 130, (K // 128, R, 4), dtype=torch.uint8, device="cuda",
                               generator=g)
        return codes, scales

    A, (codes, scales) = random(M), random(N)
    out = torch.empty(M, N, device="cuda")
    wg.forge_matmul_mxfp4(A, (codes, scales), out)
    for r in (0, 64, N // 2 - 8, N - 200, N - 72):
        rows = slice(r, r + 72)
        some = torch.empty(M, 72, device="cuda")
        wg.forge_matmul_mxfp4(A, (codes[:, rows].contiguous(), scales[:, rows].contiguous()), some)
        assert torch.equal(out[:, rows], some)
    want, size, _ = product64(torch, wg.ForgeMxfp4(*A), wg.ForgeMxfp4(
        codes[:, rows].contiguous(), scales[:, rows].contiguous()))
    assert bool(((some.double().cpu() - want).abs() <= (K / 8 + K / 64 + 2) * 2 * U * size).all())


def test_matmul_scales_by_block(env):
    """Blocks of very different scales: each lane's block takes its own scale."""
    torch, wg = env
    M, N, K = 130, 264, 512
    g = torch.Generator().manual_seed(9)
    x = torch.randn(M, K, generator=g)
    y = torch.randn(N, K, generator=g)
    ex = torch.randint(-20, 20, (M, K // 32, 1), generator=g).float()
    ey = torch.randint(-20, 20, (N, K // 32, 1), generator=g).float()
    x = (x.view(M, -1, 32) * 2.0 ** ex).view(M, K).cuda()
    y = (y.view(N, -1, 32) * 2.0 ** ey).view(N, K).cuda()
    A, B = wg.forge_mxfp4_empty(M, K), wg.forge_mxfp4_empty(N, K)
    wg.forge_quantize_mxfp4(x, rows=A)
    wg.forge_quantize_mxfp4(y, rows=B)
    out = torch.empty(M, N, device="cuda")
    wg.forge_matmul_mxfp4(A, B, out)
    check_product(torch, out, A, B)


def test_matmul_single_blocks_are_exact(env):
    """One nonzero column pair at a time: every code, sign and k position."""
    torch, wg = env
    K = 256
    vals = [0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    x = torch.zeros(K, K)
    y = torch.zeros(K, K)
    for k in range(K):
        x[k, k] = vals[k % 7] * (-1) ** k * 2.0 ** (k % 11 - 5)
        y[k, k] = vals[(k // 7) % 7] * 2.0 ** (k % 13 - 6)
    A, B = wg.forge_mxfp4_empty(K, K), wg.forge_mxfp4_empty(K, K)
    wg.forge_quantize_mxfp4(x.cuda(), rows=A)
    wg.forge_quantize_mxfp4(y.cuda(), rows=B)
    a, b = decode(torch, A)[0], decode(torch, B)[0]
    out = torch.empty(K, K, device="cuda")
    wg.forge_matmul_mxfp4(A, B, out)
    assert torch.equal(out.double().cpu(), a @ b.t())
    assert bool((a.diagonal() != 0).all()) and bool((b.diagonal() != 0).all())


def test_matmul_of_nan_blocks_and_no_columns(env):
    torch, wg = env
    x = torch.ones(64, 256, device="cuda")
    y = torch.ones(72, 256, device="cuda")
    x[5, 100], y[9, 200] = math.nan, math.inf
    A, B = wg.forge_mxfp4_empty(64, 256), wg.forge_mxfp4_empty(72, 256)
    wg.forge_quantize_mxfp4(x, rows=A)
    wg.forge_quantize_mxfp4(y, rows=B)
    out = torch.empty(64, 72, device="cuda")
    wg.forge_matmul_mxfp4(A, B, out)
    nan = torch.isnan(out.cpu())
    want = torch.zeros(64, 72, dtype=torch.bool)
    want[5], want[:, 9] = True, True
    assert torch.equal(nan, want)
    assert bool((out.cpu()[~want] == 256).all())
    empty = wg.forge_mxfp4_empty(64, 0), wg.forge_mxfp4_empty(72, 0)
    wg.forge_matmul_mxfp4(*empty, out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("T,d_in,d_out", [(1, 8, 1), (333, 264, 136), (1000, 512, 257), (0, 64, 40),
                                          (700, 1032, 300)])
def test_wgrad_adamw(env, T, d_in, d_out):
    torch, wg = env
    X = torch.randn(T, d_in, device="cuda").to(torch.bfloat16)
    dY = (torch.randn(T, (d_out + 7) // 8 * 8, device="cuda") * 0.1).to(torch.bfloat16)
    xo, yo = wg.forge_mxfp4_empty(d_in, T), wg.forge_mxfp4_empty(dY.shape[1], T)
    wg.forge_quantize_mxfp4(X, cols=xo)
    wg.forge_quantize_mxfp4(dY, cols=yo)
    # an output count that is no multiple of 8: the operand's first rows
    yo = wg.ForgeMxfp4(yo.codes[:, :d_out].contiguous(), yo.scales[:, :d_out].contiguous())
    W, m = torch.randn(d_out, d_in, device="cuda"), torch.randn(d_out, d_in, device="cuda")
    v = torch.rand(d_out, d_in, device="cuda") + 0.1
    grad = torch.empty(d_out, d_in, device="cuda")
    wg.forge_matmul_mxfp4(yo, xo, grad)
    check_product(torch, grad, yo, xo)
    for eps in (1e-8, 0.0):
        hp = dict(ADAM, eps=eps)
        ref = [t.clone() for t in (W, m, v)]
        wg.forge_adamw(grad, *ref, **hp)
        for tile in TILES:
            st = [t.clone() for t in (W, m, v)]
            wg.forge_wgrad_adamw_mxfp4(xo, yo, *st, tile=tile, **hp)
            assert all(torch.equal(a, b) for a, b in zip(st, ref)), tile


def test_linear_layer_gradients(env):
    """Y = X W^T by 4-bit products: both gradients against the same formula in
    64 bits on the decoded operands."""
    torch, wg = env
    T, d_in, d_out = 200, 136, 264
    X = torch.randn(T, d_in, device="cuda").to(torch.bfloat16)
    W = torch.randn(d_out, d_in, device="cuda") * 0.1
    dY = torch.randn(T, d_out, device="cuda").to(torch.bfloat16)
    xr, xc = both(torch, wg, X)
    wr, wc = both(torch, wg, W)
    yr, yc = both(torch, wg, dY)
    for a, b, shape in ((xr, wr, (T, d_out)), (yr, wc, (T, d_in)), (yc, xc, (d_out, d_in))):
        out = torch.empty(shape, device="cuda")
        wg.forge_matmul_mxfp4(a, b, out)
        check_product(torch, out, a, b)


def test_graph_and_streams(env):
    torch, wg = env
    T, d_in, d_out = 500, 264, 136
    X = torch.randn(T, d_in, device="cuda").to(torch.bfloat16)
    dY = torch.randn(T, d_out, device="cuda").to(torch.bfloat16)
    xo, yo = wg.forge_mxfp4_empty(d_in, T), wg.forge_mxfp4_empty(d_out, T)
    W, m = (torch.randn(d_out, d_in, device="cuda") for _ in range(2))
    v = torch.rand(d_out, d_in, device="cuda")
    ref = [t.clone() for t in (W, m, v)]

    def step(st, stream=None):
        wg.forge_quantize_mxfp4(X, cols=xo, stream=stream)
        wg.forge_quantize_mxfp4(dY, cols=yo, stream=stream)
        wg.forge_wgrad_adamw_mxfp4(xo, yo, *st, stream=stream, **ADAM)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step((W, m, v))
    for k in range(4):
        X.mul_(-1.5)
        dY.mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        step(ref)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((W, m, v), ref)), k
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step((W, m, v), stream=side)
    torch.cuda.synchronize()
    step(ref)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((W, m, v), ref))


def test_binding_refuses(env):
    torch, wg = env
    x = torch.zeros(32, 64, device="cuda")
    op = wg.forge_mxfp4_empty(32, 64)
    with pytest.raises(ValueError, match="operand of 32 rows"):
        wg.forge_quantize_mxfp4(x, cols=op)
    with pytest.raises(ValueError, match="operand of 32 rows"):
        wg.forge_quantize_mxfp4(x[:0], rows=wg.forge_mxfp4_empty(0, 64), cols=op)
    for v in (x, x[:0]):
        with pytest.raises(wg.ForgeError, match="NULL"):
            wg.forge_quantize_mxfp4(v)
    with pytest.raises(wg.ForgeError, match="ALIGN"):
        wg.forge_quantize_mxfp4(torch.zeros(32, 60, device="cuda"), rows=op)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        wg.forge_quantize_mxfp4(x.half(), rows=op)
    out = torch.zeros(32, 32, device="cuda")
    with pytest.raises(ValueError, match="padded length"):
        wg.forge_matmul_mxfp4(op, wg.forge_mxfp4_empty(32, 200), out)
    with pytest.raises(ValueError, match="scales must have shape"):
        wg.forge_matmul_mxfp4((op.codes, op.scales[:, :16].contiguous()), op, out)
    with pytest.raises(ValueError, match="on the GPU"):
        wg.forge_matmul_mxfp4(wg.forge_mxfp4_empty(32, 64, device="cpu"), op, out)
    with pytest.raises(wg.ForgeError, match="TILE"):
        wg.forge_matmul_mxfp4(op, op, out, tile=9)
    with pytest.raises(wg.ForgeError, match="CLIP"):
        wg.forge_wgrad_adamw_mxfp4(op, op, out, out.clone(), out.clone(), step=1,
                                   max_grad_norm=1.0)
    assert bool((out == 0).all())


def test_quantise_nothing(env):
    torch, wg = env
    x = torch.empty(0, 64, device="cuda")
    rows, cols = wg.forge_mxfp4_empty(0, 64), wg.forge_mxfp4_empty(64, 0)
    wg.forge_quantize_mxfp4(x, rows=rows, cols=cols)
    out = torch.ones(64, 64, device="cuda")
    wg.forge_matmul_mxfp4(cols, cols, out)
    assert bool((out == 0).all())


def test_moved_operands_are_refused_before_anything_runs(env):
    torch, wg = env

    def resized(t):
        t.untyped_storage().resize_(t.untyped_storage().nbytes() + (4 << 20))

    def data(t):
        t.data = t.clone()

    x = torch.randn(64, 256, device="cuda")
    A, B = operands(torch, wg, 64, 72, 256, 5)
    W = torch.full((64, 72), 3.0, device="cuda")
    for own, move in ((True, resized), (False, resized), (False, data)):
        for k in range(2):
            op = (wg.forge_mxfp4_empty(64, 256) if own else
                  wg.ForgeMxfp4(torch.zeros_like(A.codes), torch.zeros_like(A.scales)))
            move((op.codes, op.scales)[k])
            for call in (lambda: wg.forge_quantize_mxfp4(x, rows=op),
                         lambda: wg.forge_matmul_mxfp4(op, B, W),
                         lambda: wg.forge_matmul_mxfp4(B, op, W.t().contiguous()),
                         lambda: wg.forge_wgrad_adamw_mxfp4(B, op, W, W.clone(), W.clone(), **ADAM)):
                with pytest.raises(ValueError, match="make the operand again"):
                    call()
    assert bool((W == 3).all())


def every_epilogue(torch, wg, A, B, tiles):
    """Product and AdamW step of A B^T at each tile id, all bitwise the same; the product."""
    M, N = A.rows, B.rows
    g = torch.Generator(device="cuda").manual_seed(8)
    W, m = (torch.randn(M, N, generator=g, device="cuda") for _ in range(2))
    v = torch.rand(M, N, generator=g, device="cuda") + 0.1
    first = {}
    for tile in tiles:
        for dtype in (torch.float32, torch.bfloat16):
            guard = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
            wg.forge_matmul_mxfp4(A, B, guard[:M * N].view(M, N), tile=tile)
            assert bool((guard[M * N:] == 7).all())
            assert torch.equal(first.setdefault(dtype, guard), guard), (tile, dtype)
        st = [t.clone() for t in (W, m, v)]
        wg.forge_wgrad_adamw_mxfp4(B, A, *st, tile=tile, **ADAM)
        for a, b in zip(first.setdefault("adamw", st), st):
            assert torch.equal(a, b), tile
    out = first[torch.float32][:M * N].view(M, N)
    wg.forge_adamw(out, W, m, v, **ADAM)
    assert all(torch.equal(a, b) for a, b in zip(first["adamw"], (W, m, v)))
    assert torch.equal(first[torch.bfloat16][:M * N].view(M, N), out.to(torch.bfloat16))
    return out


@pytest.mark.parametrize("M,N,K", [(4104, 4360, 1100), (4104, 8712, 333)])
def test_more_tiles_than_workgroups(env, M, N, K):
    """306 and 595 tiles of 256x256: the persistent schedule's workers go from full to half tiles,
    from half to full ones, and through two full ones on end."""
    torch, wg = env
    A, B = operands(torch, wg, M, N, K, 12)
    out = every_epilogue(torch, wg, A, B, (4, 1, 2, 3))
    rows = sorted({0, M - 1, *range(0, M, 256), *range(255, M, 256), *range(70, M, 611)})
    some = wg.ForgeMxfp4(A.codes[:, rows].contiguous(), A.scales[:, rows].contiguous())
    check_product(torch, out[rows], some, B)


@pytest.mark.parametrize("M,N,K", [(2300, 776, 640), (520, 2056, 1100),      # 128x64 by default
                                   (300, 1032, 5000), (64, 1032, 4000),      # 64x64, slots of two stages
                                   (700, 1032, 333), (257, 520, 641)])       # 64x64
def test_tiles_of_the_librarys_own(env, M, N, K):
    torch, wg = env
    A, B = operands(torch, wg, M, N, K, 13)
    out = every_epilogue(torch, wg, A, B, (0, 2))
    check_product(torch, out, A, B)
