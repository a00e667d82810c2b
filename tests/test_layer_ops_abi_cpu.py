"""Layer norm, distillation and 8-bit block products without a GPU: bad arguments
are rejected with the documented status before any buffer is touched. Fake,
never-dereferenced pointers throughout."""
import pytest

from weight_gradient_gemm_amd import _lib, _ops

NULL = None
A, B, C, D, E, F, G, H, I = (k << 33 for k in range(1, 10))     # far apart, 16-byte aligned
NAN, INF = float("nan"), float("inf")
(OK, E_NULL, E_SHAPE, E_ALIGN, E_ALIAS, E_HPARAM, E_CLIP, E_TILE, E_DEVICE, _,
 E_DTYPE) = range(11)
F32, BF16, E4M3, E5M2 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return _ops.library()


def no_gpu():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible: valid fake pointers would launch a kernel")


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def norm(lib, x=A, xt=F32, gamma=B, beta=C, y=D, yt=BF16, mean=E, rstd=F, T=10, d=64, eps=1e-5):
    return lib.forge_layernorm(x, xt, gamma, beta, y, yt, mean, rstd, T, d, eps, None)


def back(lib, dY=A, yt=BF16, x=B, xt=F32, gamma=C, mean=D, rstd=E, dX=F, dg=G, db=H, T=10, d=64, ws=I,
         ws_bytes=1 << 20):
    return lib.forge_layernorm_backward(dY, yt, x, xt, gamma, mean, rstd, dX, dg, db, T, d, ws,
                                        ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), E_DTYPE), (dict(yt=-1), E_DTYPE), (dict(x=NULL), E_NULL), (dict(gamma=NULL), E_NULL),
    (dict(y=NULL), E_NULL), (dict(T=-1), E_SHAPE), (dict(T=(1 << 30) + 1), E_SHAPE),
    (dict(d=-8), E_SHAPE), (dict(d=65544), E_SHAPE), (dict(T=1 << 30, d=1032), E_SHAPE),
    (dict(d=60), E_ALIGN), (dict(x=A + 8), E_ALIGN), (dict(gamma=B + 4), E_ALIGN),
    (dict(beta=C + 8), E_ALIGN), (dict(y=D + 2), E_ALIGN), (dict(mean=E + 2), E_ALIGN),
    (dict(rstd=F + 1), E_ALIGN),
    (dict(y=A), E_ALIAS), (dict(y=A + 10 * 64 * 4 - 16), E_ALIAS), (dict(y=B + 64 * 4 - 16), E_ALIAS),
    (dict(y=C), E_ALIAS), (dict(mean=A + 100), E_ALIAS), (dict(rstd=E + 36), E_ALIAS),
    (dict(mean=D + 10 * 64 * 2 - 4), E_ALIAS), (dict(rstd=B), E_ALIAS),
    (dict(eps=-1e-9), E_HPARAM), (dict(eps=NAN), E_HPARAM), (dict(eps=INF), E_HPARAM),
    (dict(eps=1e39), E_HPARAM),
    (dict(T=0, x=NULL, y=NULL, gamma=NULL), OK), (dict(d=0, x=NULL, y=NULL, gamma=NULL), OK),
])
def test_layernorm_rejects(lib, kw, status):
    assert norm(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(xt=7), E_DTYPE), (dict(yt=2), E_DTYPE),
    *[({k: NULL}, E_NULL) for k in ("dY", "x", "gamma", "mean", "rstd", "dX", "dg", "ws")],
    (dict(T=-1), E_SHAPE), (dict(d=65544), E_SHAPE), (dict(ws_bytes=10 * 2 * 64 * 4 - 1), E_SHAPE),
    (dict(d=4), E_ALIGN),
    *[({k: p + 8}, E_ALIGN) for k, p in dict(dY=A, x=B, gamma=C, dX=F, dg=G, db=H, ws=I).items()],
    (dict(mean=D + 1), E_ALIGN), (dict(rstd=E + 2), E_ALIGN),
    (dict(dX=A), E_ALIAS),                                  # in place, of another type
    (dict(dX=A + 16, xt=BF16), E_ALIAS),                    # shifted
    (dict(dX=B), E_ALIAS), (dict(dg=C), E_ALIAS), (dict(db=G + 64 * 4 - 16), E_ALIAS),
    (dict(ws=A, ws_bytes=1 << 20), E_ALIAS), (dict(ws=F + 10 * 64 * 4 - 16), E_ALIAS),
    (dict(mean=I + 64), E_ALIAS), (dict(dg=E), E_ALIAS), (dict(dX=D), E_ALIAS),
    (dict(d=0, dY=NULL, x=NULL, gamma=NULL, dX=NULL, dg=NULL, ws=NULL), OK),
    (dict(T=0, dg=NULL, dY=NULL, x=NULL), E_NULL),          # zeros are still written
])
def test_layernorm_backward_rejects(lib, kw, status):
    assert back(lib, **kw) == status


def test_layernorm_workspace(lib):
    f = lib.forge_layernorm_workspace
    assert f(-1, 8) == f(8, -8) == f(1 << 31, 8) == f(8, 65544) == 0
    assert f(0, 64) >= 16 and f(10, 64) == 10 * 2 * 64 * 4 and f(1 << 20, 64) == 512 * 2 * 64 * 4


def test_layernorm_reaches_the_device_check(lib):
    no_gpu()
    assert norm(lib) == norm(lib, mean=NULL, rstd=NULL, beta=NULL) == E_DEVICE
    assert norm(lib, mean=E + 4, rstd=E + 44, eps=0.0) == E_DEVICE
    assert norm(lib, T=1 << 24, d=65536, x=1 << 45, y=1 << 46) == E_DEVICE
    assert back(lib) == back(lib, db=NULL) == back(lib, dX=A, xt=BF16) == E_DEVICE
    assert back(lib, T=0, dY=NULL, x=NULL, gamma=NULL, mean=NULL, rstd=NULL, dX=NULL) == E_DEVICE


# --------------------------------------------------------------------------
# distillation
# --------------------------------------------------------------------------
def distill(lib, z=A, zt=BF16, ld=128, u=B, ut=F32, ids=C, ib=8, w=D, loss=E, grad=F, gt=BF16, T=10,
            V=100, K=5, tau=2.0, scale=1.0, ws=G, ws_bytes=1 << 20):
    return lib.forge_distill(z, zt, ld, u, ut, ids, ib, w, loss, grad, gt, T, V, K, tau, scale, ws,
                             ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(zt=2), E_DTYPE), (dict(ut=5), E_DTYPE), (dict(gt=-1), E_DTYPE), (dict(ib=2), E_DTYPE),
    *[({k: NULL}, E_NULL) for k in ("z", "u", "ids", "loss", "ws")],
    (dict(T=-1), E_SHAPE), (dict(V=-1), E_SHAPE), (dict(K=-1), E_SHAPE), (dict(K=1025), E_SHAPE),
    (dict(V=129), E_SHAPE), (dict(ld=(1 << 22) + 8), E_SHAPE), (dict(T=(1 << 30) + 1), E_SHAPE),
    (dict(T=1 << 30, ld=2048), E_SHAPE), (dict(ws_bytes=10 * 8 + 10 * 5 * 4 - 1), E_SHAPE),
    (dict(ld=100), E_ALIGN), (dict(ids=C + 4), E_ALIGN), (dict(ids=C + 2, ib=4), E_ALIGN),
    (dict(w=D + 2), E_ALIGN), (dict(loss=E + 1), E_ALIGN),
    *[({k: p + 8}, E_ALIGN) for k, p in dict(z=A, grad=F, ws=G).items()],
    (dict(u=B + 2), E_ALIGN), (dict(u=B + 1, ut=BF16), E_ALIGN),
    (dict(grad=A, gt=F32), E_ALIAS), (dict(grad=A + 16), E_ALIAS), (dict(grad=B), E_ALIAS),
    (dict(loss=A + 10 * 128 * 2 - 4), E_ALIAS), (dict(loss=D + 36), E_ALIAS), (dict(ws=C), E_ALIAS),
    (dict(grad=G), E_ALIAS), (dict(loss=F), E_ALIAS),
    (dict(tau=0.0), E_HPARAM), (dict(tau=-1.0), E_HPARAM), (dict(tau=NAN), E_HPARAM),
    (dict(tau=INF), E_HPARAM), (dict(tau=1e-39), E_HPARAM), (dict(tau=1e39), E_HPARAM),
    (dict(scale=NAN), E_HPARAM), (dict(scale=INF), E_HPARAM), (dict(scale=1e38, tau=100.0), E_HPARAM),
    (dict(T=0, z=NULL, u=NULL, ids=NULL, w=NULL, loss=NULL, grad=NULL, ws=NULL), OK),
])
def test_distill_rejects(lib, kw, status):
    assert distill(lib, **kw) == status


def test_distill_workspace(lib):
    f = lib.forge_distill_workspace
    assert f(-1, 8, 1) == f(1, -1, 1) == f(1, 8, 1025) == f(1, (1 << 22) + 1, 1) == 0
    assert f(0, 0, 0) >= 16 and f(10, 100, 5) >= 10 * 5 * 4


def test_distill_reaches_the_device_check(lib):
    no_gpu()
    assert distill(lib) == distill(lib, grad=NULL) == distill(lib, grad=A) == E_DEVICE
    assert distill(lib, w=NULL, K=0, u=NULL, ids=NULL) == distill(lib, V=0, z=NULL) == E_DEVICE
    assert distill(lib, ib=4, ids=C + 4, loss=E + 4, w=D + 12, u=B + 4) == E_DEVICE
    assert distill(lib, ut=BF16, u=B + 2) == E_DEVICE
    assert distill(lib, scale=0.0, tau=1e-37) == distill(lib, scale=-3.0) == E_DEVICE


# --------------------------------------------------------------------------
# 8-bit operands with a scale for each block of 128
# --------------------------------------------------------------------------
def quantize(lib, x=A, xt=BF16, R=200, C=264, fmt=E4M3, square=0, rc=B, rs=C, cc=D, cs=E):
    return lib.forge_quantize_fp8_block(x, xt, R, C, fmt, square, rc, rs, cc, cs, None)


def matmul(lib, ac=A, as_=B, af=E4M3, bc=C, bs=D, bf=E4M3, out=E, M=100, N=64, Kp=256, tile=0):
    return lib.forge_matmul_fp8_block(ac, as_, af, bc, bs, bf, out, M, N, Kp, tile, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), E_DTYPE), (dict(fmt=0), E_DTYPE), (dict(fmt=1), E_DTYPE), (dict(fmt=4), E_DTYPE),
    (dict(x=NULL), E_NULL), (dict(rc=NULL), E_NULL), (dict(rs=NULL), E_NULL), (dict(cc=NULL), E_NULL),
    (dict(cs=NULL), E_NULL), (dict(rc=NULL, rs=NULL, cc=NULL, cs=NULL), E_NULL),
    (dict(R=-1), E_SHAPE), (dict(C=-8), E_SHAPE), (dict(R=(1 << 22) + 1), E_SHAPE),
    (dict(R=(1 << 30) + 1, rc=NULL, rs=NULL), E_SHAPE), (dict(C=(1 << 22) + 8, R=8), E_SHAPE),
    (dict(C=260), E_ALIGN), (dict(x=A + 8), E_ALIGN), (dict(rc=B + 8), E_ALIGN),
    (dict(rs=C + 4), E_ALIGN), (dict(cc=D + 1), E_ALIGN), (dict(cs=E + 8), E_ALIGN),
    (dict(rc=A), E_ALIAS), (dict(cs=A + 200 * 264 * 2 - 16), E_ALIAS), (dict(cc=B), E_ALIAS),
    (dict(rs=B + 200 * 384 - 16), E_ALIAS),                         # 264 columns are padded to 384
    (dict(cs=C + 3 * 256 - 16), E_ALIAS),                           # scales of 200 rows to 256
    (dict(R=0, x=NULL), OK), (dict(C=0, x=NULL), OK),
])
def test_quantize_fp8_block_rejects(lib, kw, status):
    assert quantize(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(af=0), E_DTYPE), (dict(bf=1), E_DTYPE), (dict(bf=-1), E_DTYPE),
    *[({k: NULL}, E_NULL) for k in ("ac", "as_", "bc", "bs", "out")],
    (dict(M=-1), E_SHAPE), (dict(N=-8), E_SHAPE), (dict(Kp=-128), E_SHAPE),
    (dict(M=(1 << 22) + 1), E_SHAPE), (dict(N=(1 << 22) + 8), E_SHAPE),
    (dict(Kp=(1 << 30) + 128), E_SHAPE), (dict(M=1 << 21, N=1 << 20), E_SHAPE),
    (dict(N=60), E_ALIGN), (dict(Kp=200), E_ALIGN), (dict(Kp=64), E_ALIGN),
    *[({k: p + 8}, E_ALIGN) for k, p in dict(ac=A, as_=B, bc=C, bs=D, out=E).items()],
    (dict(out=A), E_ALIAS), (dict(out=A + 100 * 256 - 16), E_ALIAS), (dict(out=D), E_ALIAS),
    (dict(out=B + 2 * 128 - 16), E_ALIAS), (dict(bs=E + 100 * 64 * 2 - 16), E_ALIAS),
    (dict(tile=-1), E_TILE), (dict(tile=5), E_TILE),
    (dict(M=0, ac=NULL, out=NULL), OK), (dict(N=0, bc=NULL, out=NULL), OK),
])
def test_matmul_fp8_block_rejects(lib, kw, status):
    assert matmul(lib, **kw) == status


def test_fp8_block_reaches_the_device_check(lib):
    no_gpu()
    assert quantize(lib) == quantize(lib, fmt=E5M2, square=1, xt=F32) == E_DEVICE
    assert quantize(lib, rc=NULL, rs=NULL) == quantize(lib, cc=NULL, cs=NULL) == E_DEVICE
    assert matmul(lib) == matmul(lib, af=E5M2, bf=E5M2, tile=4) == E_DEVICE
    assert matmul(lib, Kp=0, ac=NULL, as_=NULL, bc=NULL, bs=NULL) == E_DEVICE
    assert matmul(lib, bc=A, bs=B) == E_DEVICE                       # one operand twice


def test_operand_handles():
    import torch
    import weight_gradient_gemm_amd as wg
    cpu = wg.forge_fp8_block_empty(200, 300, device="cpu")
    assert cpu.k == 384 and tuple(cpu.codes.shape) == (6, 200, 64) and tuple(cpu.scales.shape) == (3, 256)
    assert cpu.ptrs == (cpu.codes.data_ptr(), cpu.scales.data_ptr()) and cpu._here()
    pair = wg.ForgeFp8Block(torch.zeros(6, 200, 64, dtype=torch.uint8),
                            torch.zeros(3, 256, dtype=torch.uint8), "e5m2")
    assert (pair.rows, pair.k, pair.code) == (200, 384, E5M2) and pair._here()
    pair.scales.data = pair.scales.clone()
    assert not pair._here()
    for codes, scales, err in (((6, 200, 32), (3, 256), ValueError), ((5, 200, 64), (2, 256), ValueError),
                               ((6, 200, 64), (3, 200), ValueError)):
        with pytest.raises(err):
            wg.ForgeFp8Block(torch.zeros(codes, dtype=torch.uint8), torch.zeros(scales, dtype=torch.uint8))
    with pytest.raises(TypeError):
        wg.ForgeFp8Block(torch.zeros(2, 4, 64), torch.zeros(1, 128, dtype=torch.uint8))
    with pytest.raises(ValueError, match="on the GPU"):
        _ops._fp8_operand(0, cpu, "A")
