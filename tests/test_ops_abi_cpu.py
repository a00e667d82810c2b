"""The entry points of include/forge_ops.h without a GPU: the header is C, the
library exports what it declares, the binding's struct equals the header's,
and bad arguments are rejected with the documented status before any buffer is
touched. Fake, never-dereferenced pointers throughout.
"""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from weight_gradient_gemm_amd import _lib, _ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL = None
A, B, C, D, E, F = (k << 33 for k in range(1, 7))     # far apart, 16-byte aligned
NAN, INF = float("nan"), float("inf")
(OK, E_NULL, E_SHAPE, E_ALIGN, E_ALIAS, E_HPARAM, E_CLIP, E_TILE, E_DEVICE, _,
 E_DTYPE) = range(11)
F32, BF16 = _lib.FORGE_F32, _lib.FORGE_BF16


@pytest.fixture(scope="module")
def lib():
    return _ops.library()


def declared():
    with open(os.path.join(ROOT, "include", "forge_ops.h")) as f:
        text = f.read()
    return sorted(set(re.findall(r"FORGE_API\s+[\w\s\*]*?\b(forge_\w+)\s*\(", text)))


def adam(**kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1,
                max_grad_norm=0.0)
    base.update(kw)
    return _lib.AdamWParams(*base.values())


def sgd(**kw):
    base = dict(lr=1e-3, momentum=0.9, weight_decay=0.0, max_grad_norm=0.0)
    base.update(kw)
    return _lib.SgdmParams(*base.values())


def no_gpu():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("a GPU is visible: valid fake pointers would launch a kernel")


def test_every_declared_symbol_is_exported_and_bound(lib):
    names = declared()
    assert names == sorted(_ops._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.library_path], check=True,
                         capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r"\bT (forge_\w+)", out))
    import weight_gradient_gemm_amd as wg
    for n in names:
        assert n.endswith("_workspace") or callable(getattr(wg, n))


@pytest.mark.parametrize("std", ["c99", "c11"])
def test_header_is_c(tmp_path, std):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe, lib_dir = tmp_path / "use.c", tmp_path / "use", os.path.dirname(_lib.library_path)
    src.write_text(
        "#include \"forge_ops.h\"\n#include <stddef.h>\n#include <stdio.h>\n"
        "typedef void (*fn_t)(void);\n"
        "int main(void) {\n  const fn_t fns[] = {"
        + ", ".join(f"(fn_t)&{n}" for n in declared()) + "};\n"
        "  printf(\"%d %d %d %d %d\\n\", (int)(sizeof fns / sizeof fns[0]), "
        "(int)sizeof(forge_tensor), (int)offsetof(forge_tensor, W), "
        "(int)offsetof(forge_tensor, n), (int)offsetof(forge_tensor, grad_dtype));\n"
        "  return 0;\n}\n")
    r = subprocess.run([cc, f"-std={std}", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(exe), "-L", lib_dir,
                        "-lforge", f"-Wl,-rpath,{lib_dir}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60, check=True)
    T = _ops.ForgeTensor
    assert [int(x) for x in out.stdout.split()] == [
        len(declared()), ctypes.sizeof(T), T.W.offset, T.n.offset, T.grad_dtype.offset]


# --------------------------------------------------------------------------
# global gradient norm and clipping
# --------------------------------------------------------------------------
def tensor(**kw):
    base = dict(grad=A, out=B, W=C, m=D, v=E, n=100, grad_dtype=F32)
    base.update(kw)
    return _ops.ForgeTensor(**base)


def rows(*ts):
    return (_ops.ForgeTensor * max(1, len(ts)))(*ts), len(ts)


def norm(lib, *ts, max_norm=1.0, out=F, ws=F + 4096, ws_bytes=1 << 20):
    return lib.forge_grad_norm(*rows(*ts), max_norm, out, ws, ws_bytes, None)


def test_norm_workspace_sizes(lib):
    f = lib.forge_grad_norm_workspace
    assert f(-1) == 0 and f(65537) == 0
    assert f(0) >= 16 and f(1) == f(256) == 2048 * 8 and f(257) == 2 * f(256)
    assert f(65536) == 256 * f(1)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), E_SHAPE), (dict(n=(1 << 40) + 1), E_SHAPE), (dict(grad_dtype=2), E_DTYPE),
    (dict(grad=NULL), E_NULL), (dict(grad=A + 4), E_ALIGN), (dict(grad_dtype=-1), E_DTYPE),
    (dict(grad=F), E_ALIAS), (dict(grad=F + 4096 - 16), E_ALIAS), (dict(grad=1 << 52), E_ALIGN),
])
def test_norm_rejects_tensors(lib, kw, status):
    assert norm(lib, tensor(), tensor(**kw)) == status


def test_norm_rejects(lib):
    assert norm(lib, tensor(), out=NULL) == E_NULL
    assert norm(lib, tensor(), ws=NULL) == E_NULL
    assert lib.forge_grad_norm(None, 1, 1.0, F, F + 4096, 1 << 20, None) == E_NULL
    assert lib.forge_grad_norm(None, -1, 1.0, F, F + 4096, 1 << 20, None) == E_SHAPE
    assert lib.forge_grad_norm(None, 65537, 1.0, F, F + 4096, 1 << 40, None) == E_SHAPE
    assert norm(lib, tensor(), ws_bytes=2048 * 8 - 1) == E_SHAPE
    assert norm(lib, *[tensor(n=1 << 40)] * 5) == E_SHAPE           # 5 * 2^40 > 2^42 in all
    assert norm(lib, tensor(), out=F + 2) == E_ALIGN
    assert norm(lib, tensor(), ws=F + 4096 + 8) == E_ALIGN
    assert norm(lib, tensor(), out=F + 4096) == E_ALIAS
    for bad in (-1.0, NAN, -INF):
        assert norm(lib, tensor(), max_norm=bad) == E_HPARAM


def test_steps_reject(lib):
    def clip(*ts, coef=F):
        return lib.forge_clip_grads(*rows(*ts), coef, None)

    def step(*ts, coef=F, p=None):
        return lib.forge_adamw_clipped(*rows(*ts), coef, ctypes.byref(p or adam()), None)

    def mom(*ts, coef=F, p=None):
        return lib.forge_sgdm_clipped(*rows(*ts), coef, ctypes.byref(p or sgd()), None)

    for f in (clip, step, mom):
        assert f(tensor(), coef=NULL) == E_NULL
        assert f(tensor(), coef=F + 1) == E_ALIGN
        assert f(tensor(grad=NULL)) == E_NULL
        assert f(tensor(n=-3)) == E_SHAPE
        assert f(tensor(grad_dtype=9)) == E_DTYPE
        assert f() == OK and f(tensor(n=0, grad=NULL, W=NULL, grad_dtype=77)) == OK
    assert clip(tensor(out=NULL)) == E_NULL
    assert clip(tensor(out=A + 16)) == E_ALIAS                      # shifted, not in place
    assert clip(tensor(out=A), tensor(grad=B, out=A + 384)) == E_ALIAS
    assert clip(tensor(), tensor()) == E_ALIAS                      # one output twice
    assert clip(tensor(out=F)) == E_ALIAS                           # the coefficient itself
    assert clip(tensor(grad_dtype=BF16, out=A + 192)) == E_ALIAS    # 100 * 2 bytes reach it
    for name in ("W", "m"):
        for f in (step, mom):
            assert f(tensor(**{name: NULL})) == E_NULL
            assert f(tensor(**{name: B + 8})) == E_ALIGN
            assert f(tensor(**{name: A + 384})) == E_ALIAS
            assert f(tensor(), tensor(grad=B, **{"W": B + 4096, "m": B + 8192, "v": B + 12288,
                                                 name: C})) == E_ALIAS
    assert step(tensor(v=NULL)) == E_NULL and step(tensor(v=D)) == E_ALIAS
    assert step(tensor(), p=adam(max_grad_norm=1.0)) == E_CLIP
    assert step(tensor(), p=adam(beta2=1.0)) == E_HPARAM
    assert mom(tensor(), p=sgd(max_grad_norm=1.0)) == E_CLIP
    assert mom(tensor(), p=sgd(momentum=1.0)) == E_HPARAM
    assert lib.forge_adamw_clipped(*rows(tensor()), F, None, None) == E_NULL
    assert lib.forge_sgdm_clipped(*rows(tensor()), F, None, None) == E_NULL


def test_clip_calls_reach_the_device_check(lib):
    no_gpu()
    assert norm(lib, tensor(), tensor()) == E_DEVICE                # gradients may recur
    assert norm(lib) == E_DEVICE                                    # no tensors: the norm is 0
    assert norm(lib, tensor(), max_norm=INF) == E_DEVICE
    assert lib.forge_clip_grads(*rows(tensor(out=A)), F, None) == E_DEVICE          # in place
    assert lib.forge_clip_grads(*rows(tensor(grad_dtype=BF16, out=A + 208)), F, None) == E_DEVICE
    two = rows(tensor(), tensor(W=C + 400, m=D + 400, v=E + 400))   # neighbours, one gradient
    assert lib.forge_adamw_clipped(*two, F, ctypes.byref(adam()), None) == E_DEVICE
    assert lib.forge_sgdm_clipped(*rows(tensor(v=NULL)), F, ctypes.byref(sgd()), None) == E_DEVICE


def test_tensor_list_checks():
    import torch
    import weight_gradient_gemm_amd as wg
    g = torch.zeros(4)
    with pytest.raises(ValueError, match="on the GPU"):
        wg.ForgeTensorList([g])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        wg.ForgeTensorList([g.double()])
    with pytest.raises(ValueError, match="same field"):
        wg.ForgeTensorList([], m=[], mom=[])
    with pytest.raises(ValueError, match="0 tensors|has 1 tensors"):
        wg.ForgeTensorList([], W=[g])


@pytest.fixture
def host_lists(monkeypatch):
    """Lists of CPU tensors, which no call could take, for what a call looks at first."""
    monkeypatch.setattr(_ops, "_want", lambda t, dtype, name: None)


def listed(tensors, *need):
    import torch
    try:
        return _ops._listed(torch, tensors, None, *need)
    except ValueError as e:
        return str(e)


def test_a_list_whose_tensors_moved_is_refused(host_lists):
    import torch
    import weight_gradient_gemm_amd as wg

    def make():
        # flat storages of several tensors, as well as tensors of their own, one of them empty
        return [torch.ones(n) for n in (64, 0, 7)] + list(torch.ones(96).split(32))

    def data(t):
        t.data = torch.ones_like(t)

    def resized(t):
        n = t.untyped_storage().nbytes()
        t.untyped_storage().resize_(4 * n + 1024)

    def freed(t):
        t.untyped_storage().resize_(0)

    fields = dict(out=make, W=make, m=make, v=make)
    names = ("grad", *fields)
    for move in (data, resized, freed):
        for name in names:
            for k in (0, 2, 4):
                grads, rest = make(), {n: f() for n, f in fields.items()}
                tensors = wg.ForgeTensorList(grads, **rest)
                assert listed(tensors, "out") == listed(tensors, "W", "m", "v") == (tensors.rows, 6)
                move((grads if name == "grad" else rest[name])[k])
                for need in ((), ("out",), ("W", "m"), ("W", "m", "v")):
                    got = listed(tensors, *need)
                    if name == "grad" or name in need:
                        assert "build the list again" in got and name in got, (move, name, k, need)
                    else:                                   # a field that the call does not use
                        assert got == (tensors.rows, 6)


def test_a_list_holds_its_memory(host_lists):
    # With the old storage alive nothing else can come to lie at the list's address.
    import torch
    import weight_gradient_gemm_amd as wg
    p = torch.ones(1 << 16)
    at = p.data_ptr()
    tensors = wg.ForgeTensorList([p])
    p.data = torch.empty(0)
    assert all(torch.empty(1 << 16).data_ptr() != at for _ in range(8))
    assert "build the list again" in listed(tensors)


def test_a_list_of_gradients_that_backward_replaced_is_refused(host_lists):
    import torch
    import weight_gradient_gemm_amd as wg
    W = [torch.ones(8, requires_grad=True), torch.ones(3, requires_grad=True)]

    def backward():
        sum(w.sum() for w in W).backward()

    def build(**kw):
        return wg.ForgeTensorList([w.grad for w in W], W=W, m=[torch.ones_like(w) for w in W], **kw)

    backward()
    tensors = build()
    opt = torch.optim.SGD(W)
    for again in (False, True):
        opt.zero_grad(set_to_none=False)
        backward()
        assert listed(tensors, "W", "m") == (tensors.rows, 2)        # the same gradients
    opt.zero_grad()
    assert listed(tensors, "W", "m") == (tensors.rows, 2)            # the list's are all there are
    backward()
    assert "another gradient" in listed(tensors, "W", "m") and "another" in listed(tensors)
    assert listed(build(), "W", "m")[1] == 2
    # gradients of the program's own, beside what autograd keeps
    own = wg.ForgeTensorList([torch.ones_like(w) for w in W], W=W, m=[w.grad for w in W])
    W[0].grad = torch.zeros(8)
    assert listed(own, "W")[1] == 2


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------
def lookup(lib, table=A, tt=F32, ids=B, ib=8, out=C, ot=BF16, T=10, V=100, d=64, scale=1.0):
    return lib.forge_embedding(table, tt, ids, ib, out, ot, T, V, d, scale, None)


def embgrad(lib, ids=A, ib=8, dY=B, yt=BF16, grad=C, T=10, V=100, d=64, scale=1.0, acc=0, ws=D,
            ws_bytes=1 << 20):
    return lib.forge_embedding_grad(ids, ib, dY, yt, grad, T, V, d, scale, acc, ws, ws_bytes, None)


def embadamw(lib, W=C, m=E, v=F, ws=D, p=None, T=10, V=100, d=64, ids=A, dY=B, ib=8, yt=BF16,
             scale=1.0, ws_bytes=1 << 20):
    return lib.forge_embedding_adamw(ids, ib, dY, yt, W, m, v, T, V, d, scale,
                                     ctypes.byref(p or adam()), ws, ws_bytes, None)


def embsgdm(lib, W=C, m=E, ws=D, p=None, T=10, V=100, d=64, ids=A, dY=B, ib=8, yt=BF16, scale=1.0,
            ws_bytes=1 << 20):
    return lib.forge_embedding_sgdm(ids, ib, dY, yt, W, m, T, V, d, scale,
                                    ctypes.byref(p or sgd()), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tt=2), E_DTYPE), (dict(ot=3), E_DTYPE), (dict(ib=2), E_DTYPE), (dict(ib=0), E_DTYPE),
    (dict(table=NULL), E_NULL), (dict(ids=NULL), E_NULL), (dict(out=NULL), E_NULL),
    (dict(T=-1), E_SHAPE), (dict(V=-1), E_SHAPE), (dict(d=-8), E_SHAPE),
    (dict(T=(1 << 30) + 1), E_SHAPE), (dict(V=(1 << 22) + 1), E_SHAPE),
    (dict(d=(1 << 22) + 8), E_SHAPE),
    (dict(d=60), E_ALIGN), (dict(table=A + 8), E_ALIGN), (dict(out=C + 4), E_ALIGN),
    (dict(ids=B + 4), E_ALIGN), (dict(ids=B + 2, ib=4), E_ALIGN),
    (dict(out=A), E_ALIAS), (dict(out=A + 100 * 64 * 4 - 16), E_ALIAS), (dict(out=B), E_ALIAS),
    (dict(scale=NAN), E_HPARAM), (dict(scale=INF), E_HPARAM), (dict(scale=1e39), E_HPARAM),
    (dict(T=0, ids=NULL, out=NULL), OK), (dict(d=0, table=NULL, ids=NULL, out=NULL), OK),
])
def test_embedding_rejects(lib, kw, status):
    assert lookup(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(yt=7), E_DTYPE), (dict(ib=1), E_DTYPE),
    (dict(ids=NULL), E_NULL), (dict(dY=NULL), E_NULL), (dict(ws=NULL), E_NULL),
    (dict(T=-1), E_SHAPE), (dict(V=(1 << 22) + 1), E_SHAPE), (dict(ws_bytes=100), E_SHAPE),
    (dict(d=12), E_ALIGN), (dict(dY=B + 2), E_ALIGN), (dict(ws=D + 8), E_ALIGN),
    (dict(ids=A + 4), E_ALIGN), (dict(ws=C), E_ALIAS), (dict(ws=B), E_ALIAS),
    (dict(ws=A - 64), E_ALIAS), (dict(scale=NAN), E_HPARAM),
    (dict(V=0, ws=NULL, ids=NULL, dY=NULL), OK), (dict(d=0, ws=NULL), OK),
])
def test_embedding_gradient_rejects(lib, kw, status):
    for f in (embgrad, embadamw, embsgdm):
        assert f(lib, **kw) == status, f.__name__


def test_embedding_steps_reject(lib):
    assert embgrad(lib, grad=NULL) == E_NULL and embgrad(lib, grad=C + 4) == E_ALIGN
    assert embgrad(lib, grad=B + 16) == E_ALIAS and embgrad(lib, grad=A) == E_ALIAS
    for f in (embadamw, embsgdm):
        for name in ("W", "m"):
            assert f(lib, **{name: NULL}) == E_NULL
            assert f(lib, **{name: B}) == E_ALIAS
        assert f(lib, m=C + 100 * 64 * 4 - 16) == E_ALIAS
    assert embadamw(lib, v=NULL) == E_NULL and embadamw(lib, v=E) == E_ALIAS
    assert embadamw(lib, p=adam(max_grad_norm=1.0)) == E_CLIP
    assert embadamw(lib, p=adam(step=0)) == E_HPARAM
    assert embsgdm(lib, p=sgd(max_grad_norm=INF)) == E_CLIP
    assert embsgdm(lib, p=sgd(lr=-1.0)) == E_HPARAM
    assert lib.forge_embedding_adamw(A, 8, B, BF16, C, E, F, 10, 100, 64, 1.0, None, D, 1 << 20,
                                     None) == E_NULL
    assert lib.forge_embedding_sgdm(A, 8, B, BF16, C, E, 10, 100, 64, 1.0, None, D, 1 << 20,
                                    None) == E_NULL


def test_embedding_workspace_sizes(lib):
    f = lib.forge_embedding_workspace
    for bad in ((-1, 1, 8), (1, -1, 8), (1, 1, -8), ((1 << 30) + 1, 1, 8), (1, 1 << 23, 8)):
        assert f(*bad) == 0
    assert f(0, 0, 0) >= 16
    need = f(4097, 1000, 64)
    # keys and positions twice, five tiles' digit counts, bounds, 128 chunk sums
    assert need >= 4 * 4 * 4097 + 5 * 512 * 4 + 4 * 1001 + 128 * 64 * 4
    assert f(1 << 30, 1 << 22, 1 << 22) > 0


def test_embedding_calls_reach_the_device_check(lib):
    no_gpu()
    assert lookup(lib) == E_DEVICE and lookup(lib, V=0, table=NULL) == E_DEVICE
    assert lookup(lib, out=A + 100 * 64 * 4) == E_DEVICE
    assert lookup(lib, ids=B + 4, ib=4) == E_DEVICE
    need = lib.forge_embedding_workspace(10, 100, 64)
    for f in (embgrad, embadamw, embsgdm):
        assert f(lib, ws_bytes=need) == E_DEVICE and f(lib, ws_bytes=need - 1) == E_SHAPE
        assert f(lib, T=0, ids=NULL, dY=NULL) == E_DEVICE
    assert embgrad(lib, acc=1) == E_DEVICE


# --------------------------------------------------------------------------
# microscaled 4-bit operands
# --------------------------------------------------------------------------
def quantize(lib, x=A, dt=BF16, R=100, C=256, rc=B, rs=C, cc=D, cs=E):
    return lib.forge_quantize_mxfp4(x, dt, R, C, rc, rs, cc, cs, None)


def matmul(lib, ac=A, as_=B, bc=C, bs=D, out=E, ot=F32, M=40, N=64, K=256, tile=0):
    return lib.forge_matmul_mxfp4(ac, as_, bc, bs, out, ot, M, N, K, tile, None)


G = 7 << 33


def wgrad_mx(lib, xc=A, xs=B, yc=C, ys=D, W=E, m=F, v=G, K=256, d_in=64, d_out=40, p=None,
             tile=0):
    return lib.forge_wgrad_adamw_mxfp4(xc, xs, yc, ys, W, m, v, K, d_in, d_out,
                                       ctypes.byref(p or adam()), tile, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), E_DTYPE), (dict(x=NULL), E_NULL), (dict(rc=NULL), E_NULL), (dict(rs=NULL), E_NULL),
    (dict(cc=NULL), E_NULL), (dict(cs=NULL), E_NULL),
    (dict(rc=NULL, rs=NULL, cc=NULL, cs=NULL), E_NULL),
    (dict(R=-1), E_SHAPE), (dict(C=-8), E_SHAPE), (dict(C=(1 << 22) + 8), E_SHAPE),
    (dict(R=(1 << 30) + 1), E_SHAPE), (dict(R=(1 << 22) + 1), E_SHAPE),
    (dict(R=(1 << 30) + 1, rc=NULL, rs=NULL), E_SHAPE),
    (dict(C=(1 << 30) + 8, cc=NULL, cs=NULL), E_SHAPE),
    (dict(C=100), E_ALIGN), (dict(x=A + 8), E_ALIGN), (dict(rc=B + 4), E_ALIGN),
    (dict(rs=C + 1), E_ALIGN), (dict(cc=D + 2), E_ALIGN), (dict(cs=E + 8), E_ALIGN),
    (dict(rc=A), E_ALIAS), (dict(cs=A + 100 * 256 * 2 - 16), E_ALIAS), (dict(rs=B + 16), E_ALIAS),
    (dict(cc=B), E_ALIAS), (dict(cs=D + 256 * 64 - 16), E_ALIAS),
    (dict(R=0, x=NULL), OK), (dict(C=0, x=NULL), OK),
])
def test_quantize_rejects(lib, kw, status):
    assert quantize(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=-128), E_SHAPE), (dict(K=(1 << 30) + 128), E_SHAPE), (dict(K=100), E_ALIGN),
    (dict(tile=5), E_TILE), (dict(tile=-1), E_TILE), (dict(K=130), E_ALIGN),
])
def test_products_reject(lib, kw, status):
    assert matmul(lib, **kw) == status and wgrad_mx(lib, **kw) == status


def test_matmul_rejects(lib):
    assert matmul(lib, ot=2) == E_DTYPE
    for name in ("ac", "as_", "bc", "bs", "out"):
        assert matmul(lib, **{name: NULL}) == E_NULL
        assert matmul(lib, **{name: A + (1 << 32) + 8}) == E_ALIGN
    assert matmul(lib, M=-1) == E_SHAPE and matmul(lib, N=-8) == E_SHAPE
    assert matmul(lib, M=(1 << 22) + 1) == E_SHAPE and matmul(lib, N=(1 << 22) + 8) == E_SHAPE
    assert matmul(lib, N=60) == E_ALIGN
    assert matmul(lib, out=A) == E_ALIAS and matmul(lib, out=B) == E_ALIAS
    assert matmul(lib, out=C + 64 * 128 - 16) == E_ALIAS and matmul(lib, out=D) == E_ALIAS
    assert matmul(lib, M=0, out=NULL) == OK and matmul(lib, N=0) == OK


def test_wgrad_adamw_mxfp4_rejects(lib):
    for name in ("xc", "xs", "yc", "ys", "W", "m", "v"):
        assert wgrad_mx(lib, **{name: NULL}) == E_NULL
        assert wgrad_mx(lib, **{name: A + (1 << 32) + 4}) == E_ALIGN
    assert wgrad_mx(lib, m=E) == E_ALIAS and wgrad_mx(lib, v=F + 40 * 64 * 4 - 16) == E_ALIAS
    assert wgrad_mx(lib, W=C) == E_ALIAS
    assert wgrad_mx(lib, d_in=60) == E_ALIGN
    assert wgrad_mx(lib, p=adam(max_grad_norm=1.0)) == E_CLIP
    assert wgrad_mx(lib, p=adam(eps=-1.0)) == E_HPARAM
    assert lib.forge_wgrad_adamw_mxfp4(A, B, C, D, E, F, G, 256, 64, 40, None, 0, None) == E_NULL
    assert wgrad_mx(lib, d_out=0) == OK


def test_mxfp4_calls_reach_the_device_check(lib):
    no_gpu()
    assert quantize(lib) == E_DEVICE and quantize(lib, cc=NULL, cs=NULL) == E_DEVICE
    assert quantize(lib, rc=NULL, rs=NULL, R=1 << 23) == E_DEVICE
    assert quantize(lib, cs=D + 256 * 64) == E_DEVICE            # right behind the codes
    assert matmul(lib) == E_DEVICE and matmul(lib, ot=BF16) == E_DEVICE
    assert matmul(lib, ac=A, as_=B, bc=A, bs=B) == E_DEVICE      # an operand with itself
    assert matmul(lib, K=0, ac=NULL, as_=NULL, bc=NULL, bs=NULL) == E_DEVICE
    assert wgrad_mx(lib) == E_DEVICE


def test_mxfp4_operand_shapes():
    import weight_gradient_gemm_amd as wg
    for rows, k, groups in ((3, 0, 0), (3, 1, 1), (5, 128, 1), (5, 129, 2), (8, 1000, 8)):
        op = wg.forge_mxfp4_empty(rows, k, device="cpu")
        assert (op.rows, op.k) == (rows, groups * 128)
        assert tuple(op.codes.shape) == (groups, rows, 64)
        assert tuple(op.scales.shape) == (groups, rows, 4)
        again = wg.ForgeMxfp4(op.codes, op.scales)
        assert (again.rows, again.k, again.ptrs) == (op.rows, op.k, op.ptrs)
    with pytest.raises(ValueError, match="shape"):
        wg.ForgeMxfp4(op.codes, op.scales[:1])
    with pytest.raises(TypeError, match="uint8"):
        wg.ForgeMxfp4(op.codes.int(), op.scales)
    with pytest.raises(ValueError, match="contiguous"):
        wg.ForgeMxfp4(op.codes.transpose(0, 1), op.scales)


def test_an_operand_whose_tensors_moved_is_refused():
    import torch
    import weight_gradient_gemm_amd as wg
    for make in (lambda: wg.forge_mxfp4_empty(8, 300, device="cpu"),
                 lambda: wg.ForgeMxfp4(torch.zeros(3, 8, 64, dtype=torch.uint8),
                                       torch.zeros(3, 8, 4, dtype=torch.uint8))):
        for move in ("codes", "scales"):
            op = make()
            assert _ops._operand(-1, op, "A") == (*op.ptrs, 8, 384)
            t = getattr(op, move)
            t.untyped_storage().resize_(1 << 20)
            with pytest.raises(ValueError, match="make the operand again"):
                _ops._operand(-1, op, "A")
    op, c = make(), torch.zeros(3, 8, 64, dtype=torch.uint8)
    op.codes.data = c
    with pytest.raises(ValueError, match="make the operand again"):
        _ops._operand(-1, op, "A")
    empty = wg.forge_mxfp4_empty(8, 0, device="cpu")
    assert _ops._operand(-1, empty, "A") == (None, None, 8, 0)
