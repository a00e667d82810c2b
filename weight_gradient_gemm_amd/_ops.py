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
from ._lib import FORGE_BF16, FORGE_F32, ForgeError, SgdmParams, _adamw, _torch, _want

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
    "forge_layernorm": (None, [_vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _i64, _i64, _d, _vp]),
    "forge_layernorm_workspace": (_i64, [_i64, _i64]),
    "forge_layernorm_backward": (None, [_vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                        _i64, _vp, _i64, _vp]),
    "forge_distill_workspace": (_i64, [_i64, _i64, _i64]),
    "forge_distill": (None, [_vp, _i32, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _i64, _i64,
                             _i64, _d, _d, _vp, _i64, _vp]),
    "forge_quantize_fp8_block": (None, [_vp, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "forge_matmul_fp8_block": (None, [_vp, _vp, _i32, _vp, _vp, _i32, _vp, _i64, _i64, _i64, _i32,
                                      _vp]),
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


# The small calls here take the GPU a few microseconds, so the checks are kept
# cheap: one look at the current device per call, and _lib's checks, which name
# what is wrong, only for a tensor that does not pass a short one.
def _check(status, where):
    if status:
        raise ForgeError(status, where)


_TORCH = None


def _current(stream):
    """(torch, current device, stream handle) of a call; stream None: the current one."""
    global _TORCH
    if _TORCH is None:
        _TORCH = _torch()
    torch = _TORCH
    cur = torch.cuda.current_device()
    if stream is None:
        return torch, cur, torch._C._cuda_getCurrentRawStream(cur)
    if stream.device.index != cur:
        raise ValueError(f"stream is on {stream.device} but the current device is cuda:{cur}")
    return torch, cur, stream.cuda_stream


def _in(t, dtype, name, cur):
    """The address of a contiguous tensor of `dtype` on device `cur` (None if empty)."""
    try:
        if t.dtype is dtype and t.get_device() == cur and t.is_contiguous():
            return t.data_ptr() or None
    except AttributeError:
        pass
    _want(t, dtype, name)
    return t.data_ptr() or None


def _real(torch, t, name):
    """Type code of a float32 or bfloat16 tensor."""
    dtype = getattr(t, "dtype", None)
    if dtype is torch.float32:
        return FORGE_F32
    if dtype is torch.bfloat16:
        return FORGE_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")


def _shaped(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _two(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def _workspace(torch, cur, nbytes, workspace, stream):
    """`workspace`, or one of nbytes that belongs to the stream the call runs on
    (of 16 where the sizes are out of range, for the library to say so)."""
    if workspace is not None:
        _in(workspace, torch.uint8, "workspace", cur)
        return workspace
    if stream is None:
        return torch.empty(nbytes or 16, dtype=torch.uint8, device=cur)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes or 16, dtype=torch.uint8, device=cur)


# --------------------------------------------------------------------------
# global gradient norm and clipping
# --------------------------------------------------------------------------
class ForgeTensorList:
    """Gradients, and what goes with each, of one training step: built once and
    passed to forge_grad_norm, forge_clip_grads, forge_adamw_clipped and
    forge_sgdm_clipped as often as the tensors stay where they are. A call
    raises ValueError where one of the tensors that it uses has moved
    (``p.data = ...``, a resized storage). After ``zero_grad(set_to_none=True)``,
    torch's default, backward makes new gradients, which a list of the old ones
    does not see: clear with ``set_to_none=False``, or build the list after
    every backward. A list built with weights ``W`` and their own ``grad`` as
    gradients raises where such a weight has come to another one.

    ``grads``: float32 or bfloat16 tensors of any shape, contiguous. ``out``:
    the clipped gradients' places (the gradients themselves: in place), of the
    gradients' types. ``W`` and ``m``, ``v`` (AdamW) or ``mom`` (SGD-momentum):
    float32. The list keeps the tensors and their memory alive.
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
            row.grad_dtype = _real(torch, g, "grads")
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
        # Where the tensors are. The storages are held, so that no other tensor
        # can come to lie at an address of the list.
        self._at = {name: (tuple(ts), [t.data_ptr() for t in ts])
                    for name, ts in self.tensors.items()}
        self._storages = [t.untyped_storage() for ts in self.tensors.values() for t in ts]
        self._own_grads = [(w, g) for w, g in zip(self.tensors.get("W", ()), grads)
                           if w.requires_grad and w.is_leaf and w.grad is g]
        self._norm_bytes = library().forge_grad_norm_workspace(self.count)


def _moved(name, ts, at):
    """What is wrong with a list's tensors whose addresses do not hold any more."""
    k = next(k for k, t in enumerate(ts) if t.data_ptr() != at[k])
    return ValueError(f"{name}[{k}] of the list is not where it was when the list was built "
                      "(its data was replaced or its storage resized): build the list again")


def _listed(torch, tensors, cur, *need):
    """The C array of a list that has the fields `need`, and its length."""
    if not isinstance(tensors, ForgeTensorList):
        raise TypeError(f"tensors must be a ForgeTensorList, got {type(tensors).__name__}")
    fields = tensors._at
    for name in need:
        if name not in fields:
            raise ValueError(f"the list was built without {name}")
    if tensors.device not in (None, cur):
        raise ValueError(f"the list is on cuda:{tensors.device} but the current device is "
                         f"cuda:{cur} (select it with torch.cuda.device)")
    for name in ("grad", *need):
        ts, at = fields[name]
        if list(map(torch.Tensor.data_ptr, ts)) != at:
            raise _moved(name, ts, at)
    for w, g in tensors._own_grads:
        now = w.grad
        if now is not g and now is not None and now.data_ptr() != g.data_ptr():
            raise ValueError("a weight of the list has another gradient than when the list was "
                             "built (zero_grad(set_to_none=True)?): build the list again")
    return tensors.rows, tensors.count


def _norm2(torch, cur, norm):
    p = _in(norm, torch.float32, "norm", cur)
    if norm.numel() != 2:
        raise ValueError(f"norm must hold 2 elements (norm, coefficient), got {norm.numel()}")
    return p


def forge_grad_norm(tensors, norm, *, max_norm, workspace=None, stream=None) -> None:
    """norm[0] <- the 2-norm of all gradients of the list together, norm[1] <-
    min(1, max_norm / (norm[0] + 1e-6)), the coefficient that clips to max_norm.

    ``norm`` is a float32 tensor of 2 elements; nothing is copied to the host."""
    torch, cur, st = _current(stream)
    rows, count = _listed(torch, tensors, cur)
    out = _norm2(torch, cur, norm)
    lib = library()
    ws = _workspace(torch, cur, tensors._norm_bytes, workspace, stream)
    _check(lib.forge_grad_norm(rows, count, max_norm, out, ws.data_ptr(), ws.numel(), st),
           "forge_grad_norm")


def forge_clip_grads(tensors, norm, *, stream=None) -> None:
    """out <- norm[1] * grad for every tensor of the list."""
    torch, cur, st = _current(stream)
    rows, count = _listed(torch, tensors, cur, "out")
    _check(library().forge_clip_grads(rows, count, _norm2(torch, cur, norm) + 4, st),
           "forge_clip_grads")


def forge_adamw_clipped(tensors, norm, *, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                        weight_decay=0.01, max_grad_norm=0.0, stream=None) -> None:
    """AdamW on W, m, v of every tensor of the list from norm[1] * grad."""
    torch, cur, st = _current(stream)
    rows, count = _listed(torch, tensors, cur, "W", "m", "v")
    p = _adamw(step, lr, beta1, beta2, eps, weight_decay, max_grad_norm)
    _check(library().forge_adamw_clipped(rows, count, _norm2(torch, cur, norm) + 4,
                                         ctypes.byref(p), st), "forge_adamw_clipped")


def forge_sgdm_clipped(tensors, norm, *, lr=1e-3, momentum=0.9, weight_decay=0.0,
                       max_grad_norm=0.0, stream=None) -> None:
    """SGD-momentum on W, mom of every tensor of the list from norm[1] * grad."""
    torch, cur, st = _current(stream)
    rows, count = _listed(torch, tensors, cur, "W", "m")
    p = SgdmParams(float(lr), float(momentum), float(weight_decay), float(max_grad_norm))
    _check(library().forge_sgdm_clipped(rows, count, _norm2(torch, cur, norm) + 4,
                                        ctypes.byref(p), st), "forge_sgdm_clipped")


# --------------------------------------------------------------------------
# embedding
# --------------------------------------------------------------------------
def _ids(torch, cur, ids):
    """Address, bytes of one id, and number of ids."""
    dtype = getattr(ids, "dtype", None)
    if dtype is not torch.int64 and dtype is not torch.int32:
        raise TypeError("ids must be a torch.Tensor of int32 or int64")
    return _in(ids, dtype, "ids", cur), 8 if dtype is torch.int64 else 4, ids.numel()


def forge_embedding(table, ids, out, *, scale=1.0, stream=None) -> None:
    """out[t] <- scale * table[ids[t]]; ids outside the table give rows of zeros.

    table [V, d] and out [*ids.shape, d] float32 or bfloat16, ids int32 or
    int64 of any shape."""
    torch, cur, st = _current(stream)
    ip, id_bytes, T = _ids(torch, cur, ids)
    tc, oc = _real(torch, table, "table"), _real(torch, out, "out")
    V, d = _two(table, "table")
    _shaped(out, (*ids.shape, d), "out")
    _check(library().forge_embedding(_in(table, table.dtype, "table", cur), tc, ip, id_bytes,
                                     _in(out, out.dtype, "out", cur), oc, T, V, d, scale, st),
           "forge_embedding")


def _embedding_args(ids, dY, outs, workspace, stream):
    """ids of any shape, dY [*ids.shape, d]; outs: (name, [V, d] float32) pairs.
    The leading arguments of the C calls, the outputs' addresses, sizes,
    workspace and stream."""
    torch, cur, st = _current(stream)
    ip, id_bytes, T = _ids(torch, cur, ids)
    V, d = _two(outs[0][1], outs[0][0])
    yc = _real(torch, dY, "dY")
    _shaped(dY, (*ids.shape, d), "dY")
    ptrs = []
    for name, t in outs:
        ptrs.append(_in(t, torch.float32, name, cur))
        _shaped(t, (V, d), name)
    ws = _workspace(torch, cur, library().forge_embedding_workspace(T, V, d), workspace, stream)
    return (ip, id_bytes, _in(dY, dY.dtype, "dY", cur), yc, *ptrs), (T, V, d), ws, st


def forge_embedding_grad(ids, dY, grad, *, scale=1.0, accumulate=False, workspace=None,
                         stream=None) -> None:
    """grad[r] <- scale * the sum of dY[t] over the tokens with ids[t] == r (or
    += with ``accumulate``, which leaves rows without a token alone)."""
    head, size, ws, st = _embedding_args(ids, dY, (("grad", grad),), workspace, stream)
    _check(library().forge_embedding_grad(*head, *size, scale, 1 if accumulate else 0,
                                          ws.data_ptr(), ws.numel(), st), "forge_embedding_grad")


def forge_embedding_adamw(ids, dY, W, m, v, *, step, scale=1.0, lr=1e-3, beta1=0.9, beta2=0.999,
                          eps=1e-8, weight_decay=0.01, max_grad_norm=0.0, workspace=None,
                          stream=None) -> None:
    """W, m, v <- AdamW on the embedding's gradient, in place, the gradient
    never stored; rows without a token take the step with a zero gradient."""
    head, size, ws, st = _embedding_args(ids, dY, (("W", W), ("m", m), ("v", v)), workspace,
                                         stream)
    p = _adamw(step, lr, beta1, beta2, eps, weight_decay, max_grad_norm)
    _check(library().forge_embedding_adamw(*head, *size, scale, ctypes.byref(p), ws.data_ptr(),
                                           ws.numel(), st), "forge_embedding_adamw")


def forge_embedding_sgdm(ids, dY, W, mom, *, scale=1.0, lr=1e-3, momentum=0.9, weight_decay=0.0,
                         max_grad_norm=0.0, workspace=None, stream=None) -> None:
    """W, mom <- SGD-momentum on the embedding's gradient, in place."""
    head, size, ws, st = _embedding_args(ids, dY, (("W", W), ("mom", mom)), workspace, stream)
    p = SgdmParams(float(lr), float(momentum), float(weight_decay), float(max_grad_norm))
    _check(library().forge_embedding_sgdm(*head, *size, scale, ctypes.byref(p), ws.data_ptr(),
                                          ws.numel(), st), "forge_embedding_sgdm")


# --------------------------------------------------------------------------
# microscaled 4-bit operands
# --------------------------------------------------------------------------
class ForgeMxfp4:
    """A microscaled 4-bit operand of ``rows`` rows and padded contraction
    length ``k``: uint8 ``codes`` [k / 128, rows, 64] and ``scales`` [k / 128,
    rows, 4], k a multiple of 128. It keeps its tensors and their memory alive;
    a call raises ValueError where they have moved (``codes.data = ...``, a
    resized storage)."""

    def __init__(self, codes, scales):
        torch = _torch()
        for t, name in ((codes, "codes"), (scales, "scales")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError(f"{name} must be a torch.Tensor of uint8")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if codes.dim() != 3 or codes.shape[2] != 64:
            raise ValueError("codes must have shape (groups, rows, 64), "
                             f"got {tuple(codes.shape)}")
        groups, rows, _ = codes.shape
        _shaped(scales, (groups, rows, 4), "scales")
        if scales.device != codes.device:
            raise ValueError(f"codes are on {codes.device}, scales on {scales.device}")
        self._hold, self._codes, self._scales = None, codes, scales
        self.rows, self.k, self.device = rows, groups * 128, codes.get_device()
        self.ptrs = (codes.data_ptr() or None, scales.data_ptr() or None)
        self._storages = codes.untyped_storage(), scales.untyped_storage()

    def _here(self):
        """Whether codes and scales are where the addresses point."""
        if self._hold is not None:
            return (self._hold.data_ptr() or None) == self.ptrs[0]
        return (self._codes.data_ptr() or None, self._scales.data_ptr() or None) == self.ptrs

    @property
    def codes(self):
        if self._codes is None:
            n = self.rows * self.k // 2
            self._codes = self._hold[:n].view(self.k // 128, self.rows, 64)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            n = self.rows * self.k // 2
            self._scales = self._hold[n:].view(self.k // 128, self.rows, 4)
        return self._scales


def forge_mxfp4_empty(rows, k, device=None) -> ForgeMxfp4:
    """An uninitialised operand of `rows` rows and contraction length k (padded
    to the next multiple of 128), codes and scales in one allocation."""
    torch = _torch()
    op = ForgeMxfp4.__new__(ForgeMxfp4)
    op.rows, op.k = int(rows), (int(k) + 127) // 128 * 128
    n = op.rows * op.k // 2
    op._hold = t = torch.empty(n + n // 16, dtype=torch.uint8,
                               device="cuda" if device is None else device)
    op._codes = op._scales = None
    op.device = t.get_device()
    p = t.data_ptr()
    op.ptrs = (p, p + n) if n else (None, None)
    return op


def _operand(cur, op, name):
    """Addresses of an operand's codes and scales, its rows and padded length."""
    if not isinstance(op, ForgeMxfp4):
        op = ForgeMxfp4(*op)
    if op.device != cur:
        raise ValueError(f"{name} must be on the GPU and the current device, cuda:{cur}")
    if not op._here():
        raise ValueError(f"{name}'s codes or scales are not where they were when the operand was "
                         "made (data replaced or storage resized): make the operand again")
    return *op.ptrs, op.rows, op.k


def forge_quantize_mxfp4(x, *, rows=None, cols=None, stream=None) -> None:
    """Quantises x [R, C] (float32 or bfloat16) into the operands ``rows`` (R
    rows, blocks along a row) and / or ``cols`` (C rows, blocks along a column:
    transposed)."""
    torch, cur, st = _current(stream)
    code = _real(torch, x, "x")
    xp = _in(x, x.dtype, "x", cur)
    R, C = _two(x, "x")
    ptrs = []
    for name, op, n, k in (("rows", rows, R, C), ("cols", cols, C, R)):
        if op is None:
            ptrs += (None, None)
            continue
        cp, sp, on, ok = _operand(cur, op, name)
        if on != n or ok != (k + 127) // 128 * 128:
            raise ValueError(f"{name} is an operand of {on} rows and padded length {ok}, not of "
                             f"{n} rows and length {k}")
        ptrs += (cp, sp)
    if ptrs != [None] * 4 or (rows is None and cols is None):    # else x is empty
        _check(library().forge_quantize_mxfp4(xp, code, R, C, *ptrs, st), "forge_quantize_mxfp4")


def forge_matmul_mxfp4(A, B, out, *, tile=_lib.FORGE_TILE_DEFAULT, stream=None) -> None:
    """out [M, N] (float32 or bfloat16) <- A B^T for operands A of M rows and B
    of N rows."""
    torch, cur, st = _current(stream)
    ac, as_, M, k = _operand(cur, A, "A")
    bc, bs, N, k2 = _operand(cur, B, "B")
    if k != k2:
        raise ValueError(f"A has padded length {k}, B has {k2}")
    oc = _real(torch, out, "out")
    _shaped(out, (M, N), "out")
    _check(library().forge_matmul_mxfp4(ac, as_, bc, bs, _in(out, out.dtype, "out", cur), oc, M,
                                        N, k, tile, st), "forge_matmul_mxfp4")


def forge_wgrad_adamw_mxfp4(X, dY, W, m, v, *, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                            weight_decay=0.01, max_grad_norm=0.0, tile=_lib.FORGE_TILE_DEFAULT,
                            stream=None) -> None:
    """W, m, v <- AdamW(W, m, v, g = dY^T X), in place, g never stored, from the
    operands X (d_in rows) and dY (d_out rows) over the tokens."""
    torch, cur, st = _current(stream)
    xc, xs, d_in, k = _operand(cur, X, "X")
    yc, ys, d_out, k2 = _operand(cur, dY, "dY")
    if k != k2:
        raise ValueError(f"X has padded length {k}, dY has {k2}")
    ptrs = []
    for name, t in (("W", W), ("m", m), ("v", v)):
        ptrs.append(_in(t, torch.float32, name, cur))
        _shaped(t, (d_out, d_in), name)
    p = _adamw(step, lr, beta1, beta2, eps, weight_decay, max_grad_norm)
    _check(library().forge_wgrad_adamw_mxfp4(xc, xs, yc, ys, *ptrs, k, d_in, d_out,
                                             ctypes.byref(p), tile, st),
           "forge_wgrad_adamw_mxfp4")


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def _float_or_none(torch, cur, t, shape, name):
    """Address of an optional float32 tensor of `shape`."""
    if t is None:
        return None
    p = _in(t, torch.float32, name, cur)
    _shaped(t, shape, name)
    return p


def _given(t, name):
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")


def forge_layernorm(x, gamma, beta, y, mean=None, rstd=None, *, eps=1e-5, stream=None) -> None:
    """y <- the layer norm of x over its last dimension, times gamma, plus beta.

    x and y of one shape [..., d], each float32 or bfloat16; gamma [d] and beta
    [d] (or None) float32. ``mean`` and ``rstd`` [...] float32 receive what
    forge_layernorm_backward needs."""
    torch, cur, st = _current(stream)
    xc, yc = _real(torch, x, "x"), _real(torch, y, "y")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    rows, d = x.shape[:-1], x.shape[-1]
    xp, yp = _in(x, x.dtype, "x", cur), _in(y, y.dtype, "y", cur)
    _shaped(y, x.shape, "y")
    _given(gamma, "gamma")
    _check(library().forge_layernorm(
        xp, xc, _float_or_none(torch, cur, gamma, (d,), "gamma"),
        _float_or_none(torch, cur, beta, (d,), "beta"), yp, yc,
        _float_or_none(torch, cur, mean, rows, "mean"),
        _float_or_none(torch, cur, rstd, rows, "rstd"), rows.numel(), d, eps, st),
        "forge_layernorm")


def forge_layernorm_backward(dY, x, gamma, mean, rstd, dX, dgamma, dbeta=None, *, workspace=None,
                             stream=None) -> None:
    """dX, dgamma and dbeta <- the gradients of forge_layernorm's x, gamma and beta
    from its output's dY and the mean and rstd that it stored.

    dY, x and dX of one shape [..., d], dX of x's type (and dY itself, if that is
    of x's type too); the others float32."""
    torch, cur, st = _current(stream)
    xc, yc = _real(torch, x, "x"), _real(torch, dY, "dY")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    rows, d = x.shape[:-1], x.shape[-1]
    T = rows.numel()
    ptrs = [_in(dY, dY.dtype, "dY", cur), _in(x, x.dtype, "x", cur), _in(dX, x.dtype, "dX", cur)]
    _shaped(dY, x.shape, "dY")
    _shaped(dX, x.shape, "dX")
    for t, name in ((gamma, "gamma"), (mean, "mean"), (rstd, "rstd"), (dgamma, "dgamma")):
        _given(t, name)
    lib = library()
    ws = _workspace(torch, cur, lib.forge_layernorm_workspace(T, d), workspace, stream)
    _check(lib.forge_layernorm_backward(
        ptrs[0], yc, ptrs[1], xc, _float_or_none(torch, cur, gamma, (d,), "gamma"),
        _float_or_none(torch, cur, mean, rows, "mean"),
        _float_or_none(torch, cur, rstd, rows, "rstd"), ptrs[2],
        _float_or_none(torch, cur, dgamma, (d,), "dgamma"),
        _float_or_none(torch, cur, dbeta, (d,), "dbeta"), T, d, ws.data_ptr(), ws.numel(), st),
        "forge_layernorm_backward")


# --------------------------------------------------------------------------
# distillation
# --------------------------------------------------------------------------
def forge_distill(logits, teacher, ids, loss, grad=None, *, vocab=None, weight=None, temperature=1.0,
                  scale=1.0, workspace=None, stream=None) -> None:
    """loss[t] <- scale * weight[t] * temperature^2 * KL(q_t || p_t), and grad <- its
    gradient by logits: q_t the softmax of row t's teacher logits over the
    temperature, p_t that of the student's.

    logits [..., ld] float32 or bfloat16, of which the first ``vocab`` columns (None:
    all) are the vocabulary; teacher [..., K] float32 or bfloat16 and ids [..., K]
    int32 or int64, an id outside the vocabulary (-1, say) for an entry that is not
    there; weight and loss [...] float32. ``grad`` (None: the loss alone) has the
    logits' shape, float32 or bfloat16, zeros past the vocabulary; it may be the
    logits themselves. Rows of weight 0 or without entries have loss 0 and a
    gradient of zeros."""
    torch, cur, st = _current(stream)
    zc, uc = _real(torch, logits, "logits"), _real(torch, teacher, "teacher")
    if logits.dim() < 1:
        raise ValueError("logits must have at least one dimension")
    rows, ld = logits.shape[:-1], logits.shape[-1]
    T, V = rows.numel(), ld if vocab is None else int(vocab)
    ip, id_bytes, _ = _ids(torch, cur, ids)
    if teacher.dim() < 1:
        raise ValueError("teacher must have at least one dimension")
    K = teacher.shape[-1]
    _shaped(teacher, (*rows, K), "teacher")
    _shaped(ids, (*rows, K), "ids")
    _given(loss, "loss")
    gc, gp = zc, None
    if grad is not None:
        gc = _real(torch, grad, "grad")
        _shaped(grad, logits.shape, "grad")
        gp = _in(grad, grad.dtype, "grad", cur)
    lib = library()
    ws = _workspace(torch, cur, lib.forge_distill_workspace(T, V, K), workspace, stream)
    _check(lib.forge_distill(
        _in(logits, logits.dtype, "logits", cur), zc, ld, _in(teacher, teacher.dtype, "teacher", cur),
        uc, ip, id_bytes, _float_or_none(torch, cur, weight, rows, "weight"),
        _float_or_none(torch, cur, loss, rows, "loss"), gp, gc, T, V, K, temperature, scale,
        ws.data_ptr(), ws.numel(), st), "forge_distill")


# --------------------------------------------------------------------------
# 8-bit operands with a scale for each block of 128
# --------------------------------------------------------------------------
_FP8_FORMATS = _lib._FP8


def _fp8_format(fmt):
    try:
        return _FP8_FORMATS[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"fmt must be one of {sorted(_FP8_FORMATS)}, got {fmt!r}") from None


class ForgeFp8Block:
    """An 8-bit operand with a scale for each block of 128: ``rows`` rows, padded
    contraction length ``k`` (a multiple of 128) and format ``fmt`` ("e4m3" or
    "e5m2"); uint8 ``codes`` [k / 64, rows, 64] and ``scales`` [k / 128, rows padded
    to a multiple of 128], laid out as forge_ops.h says. It keeps its tensors and
    their memory alive; a call raises ValueError where they have moved
    (``codes.data = ...``, a resized storage)."""

    def __init__(self, codes, scales, fmt="e4m3"):
        torch = _torch()
        self.fmt, self.code = fmt, _fp8_format(fmt)
        for t, name in ((codes, "codes"), (scales, "scales")):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError(f"{name} must be a torch.Tensor of uint8")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if codes.dim() != 3 or codes.shape[2] != 64 or codes.shape[0] % 2:
            raise ValueError("codes must have shape (an even number of groups, rows, 64), "
                             f"got {tuple(codes.shape)}")
        groups, rows, _ = codes.shape
        _shaped(scales, (groups // 2, (rows + 127) // 128 * 128), "scales")
        if scales.device != codes.device:
            raise ValueError(f"codes are on {codes.device}, scales on {scales.device}")
        self.codes, self.scales = codes, scales
        self.rows, self.k, self.device = rows, groups * 64, codes.get_device()
        self.ptrs = (codes.data_ptr() or None, scales.data_ptr() or None)
        self._storages = codes.untyped_storage(), scales.untyped_storage()

    def _here(self):
        """Whether codes and scales are where the addresses point."""
        return (self.codes.data_ptr() or None, self.scales.data_ptr() or None) == self.ptrs


class _Fp8BlockHeld(ForgeFp8Block):
    """An operand whose codes and scales are one allocation; their tensors are made
    when asked for."""

    def __init__(self, rows, k, fmt, device):
        torch = _TORCH or _torch()
        self.fmt, self.code = fmt, _fp8_format(fmt)
        self.rows, self.k = rows, k = int(rows), (int(k) + 127) // 128 * 128
        n = rows * k                             # a multiple of 128: scales are aligned as codes are
        self._hold = t = torch.empty(n + k // 128 * ((rows + 127) // 128 * 128), dtype=torch.uint8,
                                     device=torch.cuda.current_device() if device is None else device)
        self.device = t.get_device()
        p = t.data_ptr()
        self.ptrs = (p, p + n) if n else (None, None)

    def _here(self):
        return (self._hold.data_ptr() or None) == self.ptrs[0]

    @property
    def codes(self):
        return self._hold[:self.rows * self.k].view(self.k // 64, self.rows, 64)

    @property
    def scales(self):
        return self._hold[self.rows * self.k:].view(self.k // 128, (self.rows + 127) // 128 * 128)


def forge_fp8_block_empty(rows, k, fmt="e4m3", device=None) -> ForgeFp8Block:
    """An uninitialised operand of `rows` rows and contraction length k (padded to
    the next multiple of 128), codes and scales in one allocation."""
    return _Fp8BlockHeld(rows, k, fmt, device)


def _fp8_operand(cur, op, name):
    """An operand that is on device `cur` and has not moved."""
    if not isinstance(op, ForgeFp8Block):
        raise TypeError(f"{name} must be a ForgeFp8Block, got {type(op).__name__}")
    if op.device != cur:
        raise ValueError(f"{name} must be on the GPU and the current device, cuda:{cur}")
    if not op._here():
        raise ValueError(f"{name}'s codes or scales are not where they were when the operand was "
                         "made (data replaced or storage resized): make the operand again")
    return op


def forge_quantize_fp8_block(x, *, rows=None, cols=None, square=False, stream=None) -> None:
    """Quantises x [R, C] (float32 or bfloat16) into the operands ``rows`` (R rows,
    blocks of 128 along a row) and / or ``cols`` (C rows, blocks along a column:
    transposed), of one format. ``square``: blocks of 128 x 128, so that both hold the
    same values, as a weight's operands should."""
    torch, cur, st = _current(stream)
    code = _real(torch, x, "x")
    xp = _in(x, x.dtype, "x", cur)
    R, C = _two(x, "x")
    ptrs, fmt = [], None
    for name, op, n, k in (("rows", rows, R, C), ("cols", cols, C, R)):
        if op is None:
            ptrs += (None, None)
            continue
        op = _fp8_operand(cur, op, name)
        if op.rows != n or op.k != (k + 127) // 128 * 128:
            raise ValueError(f"{name} is an operand of {op.rows} rows and padded length {op.k}, not "
                             f"of {n} rows and length {k}")
        if fmt not in (None, op.code):
            raise ValueError(f"rows is in {rows.fmt}, cols in {cols.fmt}: one call has one format")
        fmt = op.code
        ptrs += op.ptrs
    if ptrs != [None] * 4 or (rows is None and cols is None):    # else x is empty
        _check(library().forge_quantize_fp8_block(xp, code, R, C, _lib.FORGE_FP8_E4M3 if fmt is None
                                                  else fmt, 1 if square else 0, *ptrs, st),
               "forge_quantize_fp8_block")


def forge_matmul_fp8_block(A, B, out, *, tile=_lib.FORGE_TILE_DEFAULT, stream=None) -> None:
    """out [M, N] (bfloat16) <- A B^T for operands A of M rows and B of N rows."""
    torch, cur, st = _current(stream)
    A, B = _fp8_operand(cur, A, "A"), _fp8_operand(cur, B, "B")
    if A.k != B.k:
        raise ValueError(f"A has padded length {A.k}, B has {B.k}")
    op = _in(out, torch.bfloat16, "out", cur)
    _shaped(out, (A.rows, B.rows), "out")
    _check(library().forge_matmul_fp8_block(*A.ptrs, A.code, *B.ptrs, B.code, op, A.rows, B.rows, A.k,
                                            tile, st), "forge_matmul_fp8_block")
