"""ctypes binding of the block operators of ``libgdr2.so`` (include/gdr2.h):
the norm with the residual's addition, the gated linear recurrence, and rows
in 8 bits, which these two write as activation checkpoints and read in their
gradients.

Argument marshalling only, as in ``layer``, whose conventions hold here too
(rows, packed batches, gradients, streams).  Rows in 8 bits are a ``Rows8``:

- ``codes`` float8_e4m3fn, shaped like the rows;
- ``scales`` float8_e8m0fnu [.., ceil(C / 32)], powers of two, one for 32
  columns of a row.  An element's value is its code times its block's scale.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from . import gdr2
from .gdr2 import _c_i32, _c_i64, _check, _dtype_code, _req_shape, _vp, load_library
from .layer import (KINDS, SCAN_ALGOS, _call, _empty, _grad_buffers, _mode, _offsets, _on, _packed, _raw_stream, _row_stride,
                    _rows_dtype)

ROWS8_BLOCK = 32
GLR_CHUNK = 16
GLR_ALGOS = SCAN_ALGOS
ADD_NORM_OUTPUTS = ("h", "y", "y8", "h8")
CODES, SCALES = torch.float8_e4m3fn, torch.float8_e8m0fnu

_size = ctypes.c_size_t


class Rows8(NamedTuple):
    """Rows in 8 bits (see the module's text)."""
    codes: torch.Tensor
    scales: torch.Tensor


class Rows8Args(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp)]


class PackArgs(ctypes.Structure):
    _fields_ = [("R", _c_i64), ("C", _c_i64), ("x_stride", _c_i64), ("dtype", _c_i32), ("reserved", _c_i32),
                ("x", _vp), ("out", Rows8Args)]


class UnpackArgs(ctypes.Structure):
    _fields_ = [("R", _c_i64), ("C", _c_i64), ("dtype", _c_i32), ("reserved", _c_i32), ("rows", Rows8Args), ("y", _vp)]


class AddNormArgs(ctypes.Structure):
    _fields_ = [("R", _c_i64), ("C", _c_i64), ("x_stride", _c_i64), ("res_stride", _c_i64),
                ("dtype", _c_i32), ("res_dtype", _c_i32), ("kind", _c_i32), ("eps", ctypes.c_float),
                ("x", _vp), ("residual", _vp), ("weight", _vp), ("bias", _vp), ("h", _vp), ("y", _vp),
                ("y8", Rows8Args), ("h8", Rows8Args)]


class AddNormBwdArgs(ctypes.Structure):
    _fields_ = [("R", _c_i64), ("C", _c_i64),
                ("dtype", _c_i32), ("res_dtype", _c_i32), ("kind", _c_i32), ("eps", ctypes.c_float),
                ("weight", _vp), ("h", _vp), ("h8", Rows8Args), ("dy", _vp), ("dh", _vp),
                ("dresidual", _vp), ("dx", _vp), ("dweight", _vp), ("dbias", _vp),
                ("workspace", _vp), ("workspace_bytes", _size)]


class GlrArgs(ctypes.Structure):
    _fields_ = [("B", _c_i64), ("T", _c_i64), ("C", _c_i64), ("x_stride", _c_i64), ("r_stride", _c_i64), ("i_stride", _c_i64),
                ("dtype", _c_i32), ("algo", _c_i32),
                ("x", _vp), ("r", _vp), ("i", _vp), ("A", _vp), ("h0", _vp), ("offsets", _vp),
                ("y", _vp), ("h_out", _vp), ("h_chunks", _vp), ("x8", Rows8Args), ("r8", Rows8Args), ("i8", Rows8Args),
                ("workspace", _vp), ("workspace_bytes", _size)]


class GlrStepArgs(ctypes.Structure):
    _fields_ = [("N", _c_i64), ("C", _c_i64), ("x_stride", _c_i64), ("r_stride", _c_i64), ("i_stride", _c_i64),
                ("dtype", _c_i32), ("reserved", _c_i32),
                ("state", _vp), ("x", _vp), ("r", _vp), ("i", _vp), ("A", _vp), ("y", _vp)]


class GlrBwdArgs(ctypes.Structure):
    _fields_ = [("f", GlrArgs), ("dy", _vp), ("dh_out", _vp), ("dx", _vp), ("dr", _vp), ("di", _vp), ("dA", _vp), ("dh0", _vp),
                ("workspace", _vp), ("workspace_bytes", _size)]


# entry point -> its argument struct; size queries
ENTRIES = {"gdr2_pack_rows": PackArgs, "gdr2_unpack_rows": UnpackArgs, "gdr2_add_norm_forward": AddNormArgs,
           "gdr2_add_norm_backward": AddNormBwdArgs, "gdr2_glr_forward": GlrArgs, "gdr2_glr_step": GlrStepArgs,
           "gdr2_glr_backward": GlrBwdArgs}
SIZES = {"gdr2_add_norm_backward_workspace_size": AddNormBwdArgs, "gdr2_glr_workspace_size": GlrArgs,
         "gdr2_glr_backward_workspace_size": GlrBwdArgs}

# Calls on few rows are all host time: the argument structs are packed in one
# go, and handed over as bytes.  (Those with a workspace up to its two fields.)
_GLR_STEP = struct.Struct("@5q2i6P")
_ADD_NORM = struct.Struct("@4q3if10P")
_ADD_NORM_BWD = struct.Struct("@2q3if10P")
_GLR = struct.Struct("@6q2i15P")
_GLR_BWD = struct.Struct("@6q2i16PN7P")
_WORKSPACE = struct.Struct("@PN")
_NO_WORKSPACE = bytes(_WORKSPACE.size)
assert _GLR_STEP.size == ctypes.sizeof(GlrStepArgs) and _ADD_NORM.size == ctypes.sizeof(AddNormArgs)
assert all(s.size + _WORKSPACE.size == ctypes.sizeof(a)
           for s, a in ((_ADD_NORM_BWD, AddNormBwdArgs), (_GLR, GlrArgs), (_GLR_BWD, GlrBwdArgs)))


def declare(lib):
    """Signatures of the block operators in a loaded library."""
    for name, args in ENTRIES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(args), _vp]
        f = _packed[name] = lib[name]          # a second object of the same function
        f.restype, f.argtypes = ctypes.c_int, [ctypes.c_char_p, _vp]
    for name, args in SIZES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _size, [ctypes.POINTER(args)]
        f = _packed[name] = lib[name]
        f.restype, f.argtypes = _size, [ctypes.c_char_p]
    lib.gdr2_glr_chunk_count.restype = _c_i64
    lib.gdr2_glr_chunk_count.argtypes = [_c_i64, _c_i64, ctypes.c_int]
    return lib


def _call_with_workspace(entry: str, size: str, body: bytes, workspace, like):
    """Calls an entry point with its arguments packed up to the workspace's, on
    the current stream of the device of ``like``.  The workspace's size depends
    on the device's compute units, so it is asked for with that device current."""
    index = like.device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _call_with_workspace(entry, size, body, workspace, like)
    lib = load_library()
    if workspace is None:
        need = _packed[size](body + _NO_WORKSPACE)
        if need > 0:
            workspace = like.new_empty(need, dtype=torch.uint8)
    tail = _NO_WORKSPACE
    if workspace is not None:
        tail = _WORKSPACE.pack(workspace.data_ptr(), workspace.numel() * workspace.element_size())
    status = _packed[entry](body + tail, _raw_stream(index))
    if status:
        _check(lib, status)


def _new_grads(out, like, **want):
    """``layer._grad_buffers``; where the caller gives none, fresh memory beside ``like``."""
    if out:
        return _grad_buffers(out, like.device, **want)
    return {n: None if s is None else like.new_empty(s[1], dtype=s[0]) for n, s in want.items()}


# ---- rows in 8 bits --------------------------------------------------------

def _scale_shape(shape):
    return (*shape[:-1], -(-shape[-1] // ROWS8_BLOCK))


def _new_rows8(x) -> Rows8:
    """Memory for rows like ``x`` in 8 bits."""
    return Rows8(x.new_empty(x.shape, dtype=CODES), x.new_empty(_scale_shape(x.shape), dtype=SCALES))


def _check_rows8(p, name: str, shape):
    """Dtypes and shapes of rows in 8 bits."""
    if not isinstance(p, tuple) or len(p) != 2:
        raise TypeError(f"{name} must be a Rows8 (codes, scales)")
    _req_shape(p[0], f"{name}.codes", CODES, shape)
    _req_shape(p[1], f"{name}.scales", SCALES, _scale_shape(shape))


def _rows8_args(p) -> Rows8Args:
    return Rows8Args() if p is None else Rows8Args(p[0].data_ptr(), p[1].data_ptr())


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _addrs8(rows8):
    """Pointers of several rows in 8 bits, codes and scales in turn."""
    return [t.data_ptr() for p in rows8 for t in p]


def pack_rows(x, out=None) -> Rows8:
    """Rows [.., C] in 8 bits.  ``x`` may be a column slice of wider rows.  No
    finite value is clipped; a block of 32 columns without any finite value
    keeps its infinities, beside finite ones they become NaN."""
    _rows_dtype(x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have shape (.., C), got {tuple(x.shape)}")
    C = x.shape[-1]
    ld = _row_stride(x, "x", x.dim() - 1, C)
    if out is not None:
        _check_rows8(out, "out", tuple(x.shape))
    codes, scales = (None, None) if out is None else out
    _on(x.device, (codes, scales), (x,), "out.codes out.scales x")
    if out is None:
        out = _new_rows8(x)
    _call("gdr2_pack_rows", PackArgs(x.numel() // C, C, ld, _dtype_code(x), 0, x.data_ptr(), _rows8_args(out)), x.device)
    return Rows8(*out)


def unpack_rows(rows, dtype=torch.bfloat16, out=None):
    """The values of a ``Rows8`` as rows of ``dtype`` (exact in float32)."""
    if not isinstance(rows, tuple) or len(rows) != 2 or rows[0].dim() < 1 or rows[0].shape[-1] < 1:
        raise ValueError("rows must be a Rows8 of shape (.., C)")
    shape = tuple(rows[0].shape)
    _check_rows8(rows, "rows", shape)
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    if out is not None:
        _req_shape(out, "out", dtype, shape)
    dev = rows[0].device
    _on(dev, (*rows, out), (), "rows.codes rows.scales out")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    _call("gdr2_unpack_rows", UnpackArgs(rows[0].numel() // shape[-1], shape[-1], _dtype_code(out), 0, _rows8_args(rows),
                                         out.data_ptr()), dev)
    return out


# ---- norm with the residual's addition -------------------------------------

def check_add_norm_shapes(x, residual=None, weight=None, bias=None):
    """Dtypes and shapes of the forward's inputs; returns (R, C, type of the stream)."""
    _rows_dtype(x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have shape (.., C), got {tuple(x.shape)}")
    C = x.shape[-1]
    if residual is not None:
        if residual.dtype is not x.dtype and residual.dtype is not torch.float32:
            raise TypeError(f"residual must be {x.dtype} or float32, got {residual.dtype}")
        if residual.shape != x.shape:
            raise ValueError(f"residual must have shape {tuple(x.shape)}, got {tuple(residual.shape)}")
    if weight is not None:
        _req_shape(weight, "weight", torch.float32, (C,))
    if bias is not None:
        _req_shape(bias, "bias", torch.float32, (C,))
    return x.numel() // C, C, x.dtype if residual is None else residual.dtype


def add_norm_forward(x, residual=None, weight=None, bias=None, eps: float = 1e-5, kind: str = "rms", want=("h", "y"), out=None):
    """Norm of ``h = x + residual`` over the last dimension: kind 'rms' or
    'layer'; weight, bias float32 [C].  residual has x's dtype or is float32,
    and h its dtype (x's without a residual).  Returns a dict of what ``want``
    names, None for the rest: h, the stream; y, the norm in x's dtype; y8, the
    norm as ``Rows8``; h8, the stream as ``Rows8``, which ``add_norm_backward``
    takes in place of h.  ``out``: a dict of tensors (or Rows8) to write some of
    them into; h may be written over a contiguous residual."""
    R, C, stream = check_add_norm_shapes(x, residual, weight, bias)
    code = _mode(KINDS, kind, "kind")
    for n in want:
        if n not in ADD_NORM_OUTPUTS:
            raise ValueError(f"unknown output {n!r} ({', '.join(ADD_NORM_OUTPUTS)})")
    shape, dev = x.shape, x.device
    ldx = _row_stride(x, "x", x.dim() - 1, C)
    ldr = 0 if residual is None else _row_stride(residual, "residual", x.dim() - 1, C)
    h, y, y8, h8 = _add_norm_out(out, want, tuple(shape), x.dtype, stream) if out else (None,) * 4
    _on(dev, (weight, bias, h, y, *(y8 or (None, None)), *(h8 or (None, None))) if out else (weight, bias), (x, residual),
        "weight bias h y y8.codes y8.scales h8.codes h8.scales x residual" if out else "weight bias x residual")
    if h is None and "h" in want:
        h = x.new_empty(shape, dtype=stream)
    if y is None and "y" in want:
        y = x.new_empty(shape)
    if y8 is None and "y8" in want:
        y8 = _new_rows8(x)
    if h8 is None and "h8" in want:
        h8 = _new_rows8(x)
    _call("gdr2_add_norm_forward", _ADD_NORM.pack(
        R, C, ldx, ldr, _dtype_code(x), gdr2.F32 if stream is torch.float32 else gdr2.BF16, code, eps, x.data_ptr(),
        _addr(residual), _addr(weight), _addr(bias), _addr(h), _addr(y), *((0, 0) if y8 is None else _addrs8((y8,))),
        *((0, 0) if h8 is None else _addrs8((h8,)))), dev)
    return {"h": h, "y": y, "y8": y8, "h8": h8}


def _add_norm_out(out, want, shape, dtype, stream):
    """The outputs the caller gives, of the right types and shapes: h, y, y8, h8, None for the others."""
    for n, t in out.items():
        if n not in ADD_NORM_OUTPUTS or n not in want:
            raise ValueError(f"out: {n!r} is not in want")
        if n in ("y8", "h8"):
            _check_rows8(t, f"out[{n!r}]", shape)
        else:
            _req_shape(t, f"out[{n!r}]", stream if n == "h" else dtype, shape)
    return (out.get("h"), out.get("y"), *(Rows8(*out[n]) if n in out else None for n in ("y8", "h8")))


def add_norm_backward(h, dy, dh=None, weight=None, bias=None, eps: float = 1e-5, kind: str = "rms", residual_dtype=None,
                      out=None, workspace=None):
    """Gradients of ``add_norm_forward`` for dL/dy and optionally dL/dh ``dh``
    (by the stream's other uses, in the stream's dtype).  ``h``: the stream as
    the forward returned it, or its ``Rows8``.  residual_dtype: the stream's
    dtype where neither h nor dh tells it (dy's by default).  Returns a dict:
    dresidual in the stream's dtype and dx in dy's (one tensor where the two
    are the same), dweight and dbias (float32, None without their parameter);
    ``out``: a dict of tensors to write some of them into (dresidual may be dh;
    dx only where it has a dtype of its own)."""
    _rows_dtype(dy)
    if dy.dim() < 1 or dy.shape[-1] < 1:
        raise ValueError(f"dy must have shape (.., C), got {tuple(dy.shape)}")
    C, shape, dev = dy.shape[-1], tuple(dy.shape), dy.device
    packed = isinstance(h, tuple)
    stream = h.dtype if not packed else residual_dtype or (dy.dtype if dh is None else dh.dtype)
    if stream is not dy.dtype and stream is not torch.float32:
        raise TypeError(f"the stream must be {dy.dtype} or float32, got {stream}")
    if residual_dtype is not None and residual_dtype is not stream:
        raise TypeError(f"residual_dtype is {residual_dtype}, but h is {stream}")
    if packed:
        _check_rows8(h, "h", shape)
    else:
        _req_shape(h, "h", stream, shape)
    if dh is not None:
        _req_shape(dh, "dh", stream, shape)
    for n, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _req_shape(t, n, torch.float32, (C,))
    code = _mode(KINDS, kind, "kind")
    _on(dev, (*(h if packed else (h, None)), dy, dh, weight, bias, workspace), (), "h h.scales dy dh weight bias workspace")
    param = (torch.float32, (C,))
    g = _new_grads(out, dy, dresidual=(stream, shape), dx=None if stream is dy.dtype else (dy.dtype, shape),
                      dweight=None if weight is None else param, dbias=None if bias is None else param)
    body = _ADD_NORM_BWD.pack(
        dy.numel() // C, C, _dtype_code(dy), gdr2.F32 if stream is torch.float32 else gdr2.BF16, code, eps, _addr(weight),
        *((0, *_addrs8((h,))) if packed else (h.data_ptr(), 0, 0)), dy.data_ptr(), _addr(dh), g["dresidual"].data_ptr(),
        _addr(g["dx"]), _addr(g["dweight"]), _addr(g["dbias"]))
    _call_with_workspace("gdr2_add_norm_backward", "gdr2_add_norm_backward_workspace_size", body, workspace, dy)
    if g["dx"] is None:
        g["dx"] = g["dresidual"]
    return g


# ---- gated linear recurrence -----------------------------------------------

def check_glr_shapes(x, r, i, A, offsets=None, dtype=None):
    """Dtypes and shapes of the recurrence's inputs, tensors or all three
    ``Rows8``; returns (B, T, C, shape of the rows, in 8 bits)."""
    packed = isinstance(x, tuple)
    if any(isinstance(t, tuple) != packed for t in (r, i)):
        raise TypeError("x, r and i must all be tensors or all be Rows8")
    _req_shape(A, "A", torch.float32)
    if A.dim() != 1:
        raise ValueError(f"A must have shape (C,), got {tuple(A.shape)}")
    C, lead = A.shape[0], 2 if offsets is None else 1
    rows = x[0] if packed else x
    if rows.dim() != lead + 1:
        raise ValueError(f"x must have {lead + 1} dimensions, got shape {tuple(rows.shape)}")
    shape = (*rows.shape[:-1], C)
    if packed:
        for n, t in (("x", x), ("r", r), ("i", i)):
            _check_rows8(t, n, shape)
    else:
        _rows_dtype(x)
        _req_shape(x, "x", dtype, shape)
        _req_shape(r, "r", x.dtype, shape)
        _req_shape(i, "i", x.dtype, shape)
    if offsets is not None:
        return _offsets(offsets), shape[0], C, shape, packed
    return shape[0], shape[1], C, shape, packed


def glr_chunk_count(B: int, T: int, packed: bool = False) -> int:
    """Rows of h_chunks for B sequences of T tokens (packed: T rows in all)."""
    return int(load_library().gdr2_glr_chunk_count(B, T, int(packed)))


def _chunk_rows(B: int, T: int, offsets) -> int:
    """glr_chunk_count of a call's sequences."""
    if B <= 0:
        return 0
    return B * -(-T // GLR_CHUNK) if offsets is None else T // GLR_CHUNK + B


def glr_forward(x, r, i, A, h0=None, offsets=None, out=None, h_out=None, final_state: bool = True, chunk_states=None,
                checkpoint=False, algo: str = "auto", workspace=None):
    """Gated linear recurrence.  x, r, i [B,T,C] (packed [T,C]); A float32 [C]
    (<= 0); h0 float32 [B,C].  With a = exp(A sigmoid(r)), each token makes
    h = a h + sqrt(1 - a^2) sigmoid(i) x, and y = h.  Tokens masked with r =
    -inf (or the dtype's lowest value) leave the state as it is.  Returns
    (y, h); when chunk_states is True or a float32 tensor [glr_chunk_count,C],
    (y, h, h_chunks), the state before every 16th token, which ``glr_backward``
    takes; when checkpoint is True or three Rows8 to write, (y, h, h_chunks,
    (x8, r8, i8)), the inputs in 8 bits, which it takes in their place.  h is
    the state after each sequence (None when final_state is false and no h_out
    is given; h_out may be h0)."""
    B, T, C, shape, packed = check_glr_shapes(x, r, i, A, offsets)
    if packed:
        raise TypeError("the forward takes tensors, not Rows8")
    algo = _mode(GLR_ALGOS, algo, "algo")
    for n, t in (("h0", h0), ("h_out", h_out)):
        if t is not None:
            _req_shape(t, n, torch.float32, (B, C))
    if out is not None:
        _req_shape(out, "out", x.dtype, shape)
    ck = chunk_states if isinstance(chunk_states, torch.Tensor) else None
    if ck is not None:
        _req_shape(ck, "chunk_states", torch.float32, (_chunk_rows(B, T, offsets), C))
    saved = None
    if isinstance(checkpoint, (tuple, list)):
        if len(checkpoint) != 3:
            raise ValueError("checkpoint must be True or three Rows8 (x8, r8, i8)")
        for n, t in zip(("x8", "r8", "i8"), checkpoint):
            _check_rows8(t, n, shape)
        saved = tuple(Rows8(*t) for t in checkpoint)
    lead, dev = x.dim() - 1, x.device
    flat = [t for p in saved or () for t in p]
    _on(dev, (A, h0, offsets, out, h_out, ck, workspace, *flat), (x, r, i),
        "A h0 offsets out h_out chunk_states workspace " + "x8 x8.scales r8 r8.scales i8 i8.scales " * bool(flat) + "x r i")
    out = _empty(out, x.shape, x)
    if h_out is None and final_state:
        h_out = A.new_empty((B, C))
    if ck is None and (chunk_states or checkpoint):
        ck = A.new_empty((_chunk_rows(B, T, offsets), C))
    if saved is None and checkpoint:
        saved = tuple(_new_rows8(x) for _ in range(3))
    body = _GLR.pack(B, T, C, _row_stride(x, "x", lead, C), _row_stride(r, "r", lead, C), _row_stride(i, "i", lead, C),
                     _dtype_code(x), algo, x.data_ptr(), r.data_ptr(), i.data_ptr(), A.data_ptr(), _addr(h0), _addr(offsets),
                     out.data_ptr(), _addr(h_out), _addr(ck), *(_addrs8(saved) if saved else (0,) * 6))
    _call_with_workspace("gdr2_glr_forward", "gdr2_glr_workspace_size", body, workspace, x)
    if saved is not None:
        return out, h_out, ck, saved
    return (out, h_out) if ck is None else (out, h_out, ck)


def glr_step(state, x, r, i, A, out=None):
    """The recurrence for one token of each of N sequences, in place on
    ``state`` float32 [N,C]; x, r, i [N,C].  Returns y [N,C]."""
    if x.dim() != 2:
        raise ValueError(f"x must have shape (N, C), got {tuple(x.shape)}")
    (N, C), e = x.shape, x.dtype
    if not (A.shape == (C,) and A.dtype is torch.float32 and (e is torch.bfloat16 or e is torch.float32) and r.dtype is e
            and i.dtype is e and r.shape == x.shape == i.shape and state.dtype is torch.float32 and state.shape == x.shape):
        _rows_dtype(x)
        _req_shape(A, "A", torch.float32, (C,))
        _req_shape(r, "r", e, (N, C))
        _req_shape(i, "i", e, (N, C))
        _req_shape(state, "state", torch.float32, (N, C))
    if out is not None:
        _req_shape(out, "out", e, (N, C))
    dev = x.device
    _on(dev, (state, A, out), (x, r, i), "state A out x r i")
    out = _empty(out, (N, C), x)
    _call("gdr2_glr_step", _GLR_STEP.pack(N, C, _row_stride(x, "x", 1, C), _row_stride(r, "r", 1, C), _row_stride(i, "i", 1, C),
                                          _dtype_code(x), 0, state.data_ptr(), x.data_ptr(), r.data_ptr(), i.data_ptr(),
                                          A.data_ptr(), out.data_ptr()), dev)
    return out


def glr_backward(x, r, i, A, dy, h_chunks, offsets=None, dh_out=None, want_dh0: bool = True, algo: str = "auto", out=None,
                 workspace=None):
    """Gradients of ``glr_forward`` for dL/dy and optionally dL/dh ``dh_out``
    float32 [B,C]; x, r, i the forward's, or the Rows8 it wrote; h_chunks as
    the forward of the same inputs returned them.  Returns a dict: dx, dr, di
    in dy's dtype; dA, dh0 float32; ``out``: a dict of tensors to write some of
    them into (dh0 may be dh_out)."""
    B, T, C, shape, packed = check_glr_shapes(x, r, i, A, offsets)
    _rows_dtype(dy)
    _req_shape(dy, "dy", None if packed else x.dtype, shape)
    _req_shape(h_chunks, "h_chunks", torch.float32, (_chunk_rows(B, T, offsets), C))
    if dh_out is not None:
        _req_shape(dh_out, "dh_out", torch.float32, (B, C))
    algo = _mode(GLR_ALGOS, algo, "algo")
    dev, lead = dy.device, dy.dim() - 1
    dense = (*x, *r, *i) if packed else (None,) * 6
    _on(dev, (A, offsets, dy, h_chunks, dh_out, workspace, *dense), () if packed else (x, r, i),
        "A offsets dy h_chunks dh_out workspace x x.scales r r.scales i i.scales x r i")
    rows = (dy.dtype, shape)
    g = _new_grads(out, dy, dx=rows, dr=rows, di=rows, dA=(torch.float32, (C,)),
                      dh0=(torch.float32, (B, C)) if want_dh0 else None)
    if packed:
        strides, given = (0, 0, 0), (0, 0, 0)
    else:
        strides = _row_stride(x, "x", lead, C), _row_stride(r, "r", lead, C), _row_stride(i, "i", lead, C)
        given = x.data_ptr(), r.data_ptr(), i.data_ptr()
    body = _GLR_BWD.pack(B, T, C, *strides, _dtype_code(dy), algo, *given, A.data_ptr(), 0, _addr(offsets), 0, 0, h_chunks.data_ptr(),
                         *(_addrs8((x, r, i)) if packed else (0,) * 6), 0, 0, dy.data_ptr(), _addr(dh_out), g["dx"].data_ptr(),
                         g["dr"].data_ptr(), g["di"].data_ptr(), g["dA"].data_ptr(), _addr(g["dh0"]))
    _call_with_workspace("gdr2_glr_backward", "gdr2_glr_backward_workspace_size", body, workspace, dy)
    return g
