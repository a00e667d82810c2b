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
