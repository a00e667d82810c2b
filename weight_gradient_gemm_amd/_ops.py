"""ctypes binding of the entry points of include/forge_ops.h; argument
marshalling only, in the manner of _lib: torch tensors on the current HIP
device, sizes read off them, everything else validated by the library.

A call that needs a workspace takes one from torch's allocator, on the stream
it runs on, unless the caller passes its own (``workspace``, a uint8 tensor):
then two calls that may run at the same time need two.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import (SgdmParams, _adamw, _check, _dtype_code, _ptr, _stream,
                   _torch, _want)

_i32, _i64, _vp, _d = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_double
_adam_p = ctypes.POINTER(_lib.AdamWParams)
_sgdm_p = ctypes.POINTER(_lib.SgdmParams)


class ForgeTensor(ctypes.Structure):
    """forge_tensor of the C header."""
    _fields_ = [("grad", _vp), ("out", _vp), ("W", _vp), ("m", _vp), ("v", _vp), ("n", _i64),
                ("grad_dtype", _i32)]


_list_p = ctypes.POINTER(ForgeTensor)

# Result type (None: a status) and arguments of each entry point.
_SIGNATURES = {
    "forge_grad_norm_workspace": (_i64, [_i32]),
    "forge_grad_norm": (None, [_list_p, _i32, _d, _vp, _vp, _i64, _vp]),
    "forge_clip_grads": (None, [_list_p, _i32, _vp, _vp]),
    "forge_adamw_clipped": (None, [_list_p, _i32, _vp, _adam_p, _vp]),
    "forge_sgdm_clipped": (None, [_list_p, _i32, _vp, _sgdm_p, _vp]),
    "forge_embedding": (None, [_vp, _i32, _vp, _i32, _vp, _i32, _i64, _i64, _i64, _d, _vp]),
    "forge_embedding_workspace": (_i64, [_i64, _i64, _i64]),
    "forge_embedding_grad": (None, [_vp, _i32, _vp, _i32, _vp, _i64, _i64, _i64, _d, _i32, _vp,
                                    _i64, _vp]),
    "forge_embedding_adamw": (None, [_vp, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _d,
                                     _adam_p, _vp, _i64, _vp]),
    "forge_embedding_sgdm": (None, [_vp, _i32, _vp, _i32, _vp, _vp, _i64, _i64, _i64, _d, _sgdm_p,
                                    _vp, _i64, _vp]),
    "forge_quantize_mxfp4": (None, [_vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "forge_matmul_mxfp4": (None, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i32, _vp]),
    "forge_wgrad_adamw_mxfp4": (None, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                       _adam_p, _i32, _vp]),
}

_DONE = None


def library() -> ctypes.CDLL:
    """The loaded libforge.so with the signatures of forge_ops.h."""
    global _DONE
    lib = _lib.library()
    if _DONE is not lib:
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res or _i32, args
        _DONE = lib
    return lib


def _workspace(nbytes, workspace, stream):
    """`workspace`, or one of nbytes that belongs to the stream the call runs on."""
    torch = _torch()
    if workspace is not None:
        _want(workspace, torch.uint8, "workspace")
        return workspace
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------
# global gradient norm and clipping
# --------------------------------------------------------------------------
class ForgeTensorList:
    """Gradients, and what goes with each, of one training step: built once and
    passed to forge_grad_norm, forge_clip_grads, forge_adamw_clipped and
    forge_sgdm_clipped as often as the tensors stay where they are.

    ``grads``: float32 or bfloat16 tensors of any shape, contiguous. ``out``:
    the clipped gradients' places (the gradients themselves: in place), of the
    gradients' types. ``W`` and ``m``, ``v`` (AdamW) or ``mom`` (SGD-momentum):
    float32. The list keeps the tensors alive.
    """

    def __init__(self, grads, *, out=None, W=None, m=None, v=None, mom=None):
        torch = _torch()
        if m is not None and mom is not None:
            raise ValueError("m (AdamW) and mom (SGD-momentum) are the same field: give one")
        grads = list(grads)
        fields = {"out": out, "W": W, "m": m if mom is None else mom, "v": v}
        self.tensors = {"grad": grads}
        rows = (ForgeTensor * max(1, len(grads)))()
        for row, g in zip(rows, grads):
            if not isinstance(g, torch.Tensor):
                raise TypeError("grads must be torch.Tensors")
            row.grad_dtype = _dtype_code(g, "grads")
            _want(g, g.dtype, "grads")
            row.grad, row.n = g.data_ptr() or None, g.numel()
        for name, ts in fields.items():
            if ts is None:
                continue
            ts = list(ts)
            if len(ts) != len(grads):
                raise ValueError(f"{name} has {len(ts)} tensors, grads has {len(grads)}")
            for row, g, t in zip(rows, grads, ts):
                _want(t, g.dtype if name == "out" else torch.float32, name)
                if t.numel() != g.numel():
                    raise ValueError(f"{name} has a tensor of {t.numel()} elements where the "
                                     f"gradient has {g.numel()}")
                setattr(row, name, t.data_ptr() or None)
            self.tensors[name] = ts
        self.rows, self.count = rows, len(grads)
        self.device = grads[0].device.index if grads else None

    def _args(self, *need):
        for name in need:
            if name not in self.tensors:
                raise ValueError(f"the list was built without {name}")
        cur = _torch().cuda.current_device()
        if self.device not in (None, cur):
            raise ValueError(f"the list is on cuda:{self.device} but the current device is "
                             f"cuda:{cur} (select it with torch.cuda.device)")
        return self.rows, self.count


def _norm2(norm):
    _want(norm, _torch().float32, "norm")
    if norm.numel() != 2:
        raise ValueError(f"norm must hold 2 elements (norm, coefficient), got {norm.numel()}")
    return norm.data_ptr()


def forge_grad_norm(tensors, norm, *, max_norm, workspace=None, stream=None) -> None:
    """norm[0] <- the 2-norm of all gradients of the list together, norm[1] <-
    min(1, max_norm / (norm[0] + 1e-6)), the coefficient that clips to max_norm.

    ``norm`` is a float32 tensor of 2 elements; nothing is copied to the host."""
    rows, count = tensors._args()
    out = _norm2(norm)
    lib = library()
    ws = _workspace(lib.forge_grad_norm_workspace(count), workspace, stream)
    _check(lib.forge_grad_norm(rows, count, float(max_norm), out, _ptr(ws), ws.numel(),
                               _stream(stream)), "forge_grad_norm")


def forge_clip_grads(tensors, norm, *, stream=None) -> None:
    """out <- norm[1] * grad for every tensor of the list."""
    rows, count = tensors._args("out")
    _check(library().forge_clip_grads(rows, count, _norm2(norm) + 4, _stream(stream)),
           "forge_clip_grads")


def forge_adamw_clipped(tensors, norm, *, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                        weight_decay=0.01, max_grad_norm=0.0, stream=None) -> None:
    """AdamW on W, m, v of every tensor of the list from norm[1] * grad."""
    rows, count = tensors._args("W", "m", "v")
    p = _adamw(step, lr, beta1, beta2, eps, weight_decay, max_grad_norm)
    _check(library().forge_adamw_clipped(rows, count, _norm2(norm) + 4, ctypes.byref(p),
                                         _stream(stream)), "forge_adamw_clipped")


def forge_sgdm_clipped(tensors, norm, *, lr=1e-3, momentum=0.9, weight_decay=0.0,
                       max_grad_norm=0.0, stream=None) -> None:
    """SGD-momentum on W, mom of every tensor of the list from norm[1] * grad."""
    rows, count = tensors._args("W", "m")
    p = SgdmParams(float(lr), float(momentum), float(weight_decay), float(max_grad_norm))
    _check(library().forge_sgdm_clipped(rows, count, _norm2(norm) + 4, ctypes.byref(p),
                                        _stream(stream)), "forge_sgdm_clipped")


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------
def _ids(ids):
    torch = _torch()
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be a torch.Tensor of int32 or int64")
    _want(ids, ids.dtype, "ids")
    return ids.numel(), ids.element_size()


def _rows_like(t, shape, name, dtype=None):
    code = _dtype_code(t, name) if dtype is None else None
    _want(t, dtype or t.dtype, name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return code


def forge_embedding(table, ids, out, *, scale=1.0, stream=None) -> None:
    """out[t] <- scale * table[ids[t]]; ids outside the table give rows of zeros.

    table [V, d] and out [*ids.shape, d] float32 or bfloat16, ids int32 or
    int64 of any shape."""
    T, id_bytes = _ids(ids)
    V, d = _lib._shape2(table, "table")
    tc = _rows_like(table, (V, d), "table")
    oc = _rows_like(out, (*ids.shape, d), "out")
    _check(library().forge_embedding(_ptr(table), tc, _ptr(ids), id_bytes, _ptr(out), oc, T, V, d,
                                     float(scale), _stream(stream)), "forge_embedding")


def _embedding_args(ids, dY, outs, workspace, stream):
    """ids of any shape, dY [*ids.shape, d]; outs: (name, [V, d] float32) pairs."""
    T, id_bytes = _ids(ids)
    V, d = _lib._shape2(outs[0][1], outs[0][0])
    yc = _rows_like(dY, (*ids.shape, d), "dY")
    for name, t in outs:
        _rows_like(t, (V, d), name, _torch().float32)
    ws = _workspace(library().forge_embedding_workspace(T, V, d), workspace, stream)
    return (_ptr(ids), id_bytes, _ptr(dY), yc), (T, V, d), ws


def forge_embedding_grad(ids, dY, grad, *, scale=1.0, accumulate=False, workspace=None,
                         stream=None) -> None:
    """grad[r] <- scale * the sum of dY[t] over the tokens with ids[t] == r (or
    += with ``accumulate``, which leaves rows without a token alone)."""
    head, (T, V, d), ws = _embedding_args(ids, dY, (("grad", grad),), workspace, stream)
    _check(library().forge_embedding_grad(*head, _ptr(grad), T, V, d, float(scale),
                                          int(bool(accumulate)), _ptr(ws), ws.numel(),
                                          _stream(stream)), "forge_embedding_grad")


def forge_embedding_adamw(ids, dY, W, m, v, *, step, scale=1.0, lr=1e-3, beta1=0.9, beta2=0.999,
                          eps=1e-8, weight_decay=0.01, max_grad_norm=0.0, workspace=None,
                          stream=None) -> None:
    """W, m, v <- AdamW on the embedding's gradient, in place, the gradient
    never stored; rows without a token take the step with a zero gradient."""
    head, (T, V, d), ws = _embedding_args(ids, dY, (("W", W), ("m", m), ("v", v)), workspace,
                                          stream)
    p = _adamw(step, lr, beta1, beta2, eps, weight_decay, max_grad_norm)
    _check(library().forge_embedding_adamw(*head, _ptr(W), _ptr(m), _ptr(v), T, V, d,
                                           float(scale), ctypes.byref(p), _ptr(ws), ws.numel(),
                                           _stream(stream)), "forge_embedding_adamw")


def forge_embedding_sgdm(ids, dY, W, mom, *, scale=1.0, lr=1e-3, momentum=0.9, weight_decay=0.0,
                         max_grad_norm=0.0, workspace=None, stream=None) -> None:
    """W, mom <- SGD-momentum on the embedding's gradient, in place."""
    head, (T, V, d), ws = _embedding_args(ids, dY, (("W", W), ("mom", mom)), workspace, stream)
    p = SgdmParams(float(lr), float(momentum), float(weight_decay), float(max_grad_norm))
    _check(library().forge_embedding_sgdm(*head, _ptr(W), _ptr(mom), T, V, d, float(scale),
                                          ctypes.byref(p), _ptr(ws), ws.numel(),
                                          _stream(stream)), "forge_embedding_sgdm")


# --------------------------------------------------------------------------
# microscaled 4-bit operands
# --------------------------------------------------------------------------
def forge_mxfp4_empty(rows, k, device=None):
    """(codes, scales), uninitialised, of an operand of `rows` rows and
    contraction length k: uint8 [rows, Kp / 2] and [Kp / 128, rows, 4], Kp the
    next multiple of 128."""
    torch = _torch()
    groups = (int(k) + 127) // 128
    device = "cuda" if device is None else device
    return (torch.empty((int(rows), groups * 64), dtype=torch.uint8, device=device),
            torch.empty((groups, int(rows), 4), dtype=torch.uint8, device=device))


def _operand(pair, name):
    """Checked (codes, scales) of an operand; its rows and padded length."""
    torch = _torch()
    codes, scales = pair
    _want(codes, torch.uint8, f"{name} codes")
    _want(scales, torch.uint8, f"{name} scales")
    rows, half = _lib._shape2(codes, f"{name} codes")
    if half % 64:
        raise ValueError(f"{name} codes must have a multiple of 64 columns, got {half}")
    if tuple(scales.shape) != (half // 64, rows, 4):
        raise ValueError(f"{name} scales must have shape {(half // 64, rows, 4)}, "
                         f"got {tuple(scales.shape)}")
    return rows, half * 2


def forge_quantize_mxfp4(x, *, rows=None, cols=None, stream=None) -> None:
    """Quantises x [R, C] (float32 or bfloat16) into the operands ``rows`` (R
    rows, blocks along a row) and / or ``cols`` (C rows, blocks along a column:
    transposed), each a pair as forge_mxfp4_empty makes."""
    R, C = _lib._shape2(x, "x")
    code = _rows_like(x, (R, C), "x")
    ptrs = []
    for name, pair, want in (("rows", rows, (R, C)), ("cols", cols, (C, R))):
        if pair is None:
            ptrs += [None, None]
            continue
        n, k = _operand(pair, name)
        if (n, k) != (want[0], (want[1] + 127) // 128 * 128):
            raise ValueError(f"{name} is an operand of {n} rows and padded length {k}, not of "
                             f"{want[0]} rows and length {want[1]}")
        if n and k:
            ptrs += [_ptr(pair[0]), _ptr(pair[1])]
        else:
            return                           # x is empty: nothing to write
    _check(library().forge_quantize_mxfp4(_ptr(x), code, R, C, *ptrs, _stream(stream)),
           "forge_quantize_mxfp4")


def forge_matmul_mxfp4(A, B, out, *, tile=_lib.FORGE_TILE_DEFAULT, stream=None) -> None:
    """out [M, N] (float32 or bfloat16) <- A B^T for operands A of M rows and B
    of N rows, each a (codes, scales) pair."""
    M, k = _operand(A, "A")
    N, k2 = _operand(B, "B")
    if k != k2:
        raise ValueError(f"A has padded length {k}, B has {k2}")
    oc = _rows_like(out, (M, N), "out")
    _check(library().forge_matmul_mxfp4(_ptr(A[0]), _ptr(A[1]), _ptr(B[0]), _ptr(B[1]), _ptr(out),
                                        oc, M, N, k, int(tile), _stream(stream)),
           "forge_matmul_mxfp4")


def forge_wgrad_adamw_mxfp4(X, dY, W, m, v, *, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                            weight_decay=0.01, max_grad_norm=0.0, tile=_lib.FORGE_TILE_DEFAULT,
                            stream=None) -> None:
    """W, m, v <- AdamW(W, m, v, g = dY^T X), in place, g never stored, from the
    operands X (d_in rows) and dY (d_out rows) over the tokens."""
    d_in, k = _operand(X, "X")
    d_out, k2 = _operand(dY, "dY")
    if k != k2:
        raise ValueError(f"X has padded length {k}, dY has {k2}")
    _lib._state_like(W, (("m", m), ("v", v)), d_out, d_in)
    p = _adamw(step, lr, beta1, beta2, eps, weight_decay, max_grad_norm)
    _check(library().forge_wgrad_adamw_mxfp4(_ptr(X[0]), _ptr(X[1]), _ptr(dY[0]), _ptr(dY[1]),
                                             _ptr(W), _ptr(m), _ptr(v), k, d_in, d_out,
                                             ctypes.byref(p), int(tile), _stream(stream)),
           "forge_wgrad_adamw_mxfp4")
