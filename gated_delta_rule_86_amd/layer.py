"""ctypes binding of the layer operators of ``libgdr2.so`` (include/gdr2.h):
the short causal convolution, the selective state space scan and the norms
that stand around the recurrence in a sequence-mixing layer.

Argument marshalling only, as in ``gdr2``.  Common to all functions:

- rows are float32 or bfloat16; weights, biases, A, skip and every state of
  the scan are float32.  A row input may be a column slice of a wider
  projection (last dimension dense, equally spaced rows); everything else is
  contiguous.
- a batch is dense, ``[B, T, ...]``, or packed: ``[T, ...]`` with ``offsets``,
  an int64 device tensor of ``B + 1`` ascending row numbers (sequences may be
  empty).  Rows of no sequence are not touched, in gradients neither: in a
  result the call allocates they hold what the memory held before.  Pass
  ``out`` where that matters (zeros, for a padded batch that is trained on).
- gradients of rows have the rows' dtype, gradients of parameters and states
  are float32.
- the call is enqueued on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import gdr2
from .gdr2 import _c_i32, _c_i64, _check, _dtype_code, _ptr, _req_dev, _req_shape, _vp, load_library

ACTIVATIONS = {None: 0, "silu": 1}
KINDS = {"layer": 0, "rms": 1}
SCAN_ALGOS = {n: gdr2.ALGOS[n] for n in ("auto", "staged", "segmented")}
SCAN_SOFTPLUS = 1
SCAN_CHUNK = 32

_size = ctypes.c_size_t


class ConvArgs(ctypes.Structure):
    _fields_ = [("B", _c_i64), ("T", _c_i64), ("C", _c_i64), ("x_stride", _c_i64),
                ("width", _c_i32), ("dtype", _c_i32), ("act", _c_i32), ("reserved", _c_i32),
                ("x", _vp), ("weight", _vp), ("bias", _vp), ("state0", _vp), ("offsets", _vp),
                ("y", _vp), ("state_out", _vp)]


class ConvStepArgs(ctypes.Structure):
    _fields_ = [("N", _c_i64), ("C", _c_i64), ("x_stride", _c_i64),
                ("width", _c_i32), ("dtype", _c_i32), ("act", _c_i32), ("reserved", _c_i32),
                ("state", _vp), ("x", _vp), ("weight", _vp), ("bias", _vp), ("y", _vp)]


class ConvBwdArgs(ctypes.Structure):
    _fields_ = [("B", _c_i64), ("T", _c_i64), ("C", _c_i64), ("x_stride", _c_i64),
                ("width", _c_i32), ("dtype", _c_i32), ("act", _c_i32), ("reserved", _c_i32),
                ("x", _vp), ("weight", _vp), ("bias", _vp), ("state0", _vp), ("offsets", _vp),
                ("dy", _vp), ("dstate", _vp), ("dx", _vp), ("dweight", _vp), ("dbias", _vp), ("dstate0", _vp),
                ("workspace", _vp), ("workspace_bytes", _size)]


class ScanArgs(ctypes.Structure):
    _fields_ = [("B", _c_i64), ("T", _c_i64), ("C", _c_i64), ("N", _c_i64), ("G", _c_i64),
                ("x_stride", _c_i64), ("dt_stride", _c_i64), ("b_stride", _c_i64), ("c_stride", _c_i64),
                ("z_stride", _c_i64),
                ("dtype", _c_i32), ("flags", _c_i32), ("algo", _c_i32), ("reserved", _c_i32),
                ("x", _vp), ("dt", _vp), ("Bt", _vp), ("Ct", _vp), ("z", _vp),
                ("A", _vp), ("skip", _vp), ("dt_bias", _vp), ("h0", _vp), ("offsets", _vp),
                ("y", _vp), ("h_out", _vp), ("h_chunks", _vp), ("workspace", _vp), ("workspace_bytes", _size)]


class ScanStepArgs(ctypes.Structure):
    _fields_ = [("s", ScanArgs), ("state", _vp)]


class ScanBwdArgs(ctypes.Structure):
    _fields_ = [("f", ScanArgs), ("dy", _vp), ("dh_out", _vp),
                ("dx", _vp), ("ddt", _vp), ("dBt", _vp), ("dCt", _vp), ("dz", _vp),
                ("dA", _vp), ("dskip", _vp), ("ddt_bias", _vp), ("dh0", _vp),
                ("workspace", _vp), ("workspace_bytes", _size)]


class NormArgs(ctypes.Structure):
    _fields_ = [("R", _c_i64), ("C", _c_i64), ("x_stride", _c_i64), ("z_stride", _c_i64),
                ("dtype", _c_i32), ("kind", _c_i32), ("eps", ctypes.c_float), ("reserved", _c_i32),
                ("x", _vp), ("z", _vp), ("weight", _vp), ("bias", _vp), ("y", _vp)]


class NormBwdArgs(ctypes.Structure):
    _fields_ = [("f", NormArgs), ("dy", _vp), ("dx", _vp), ("dz", _vp), ("dweight", _vp), ("dbias", _vp),
                ("workspace", _vp), ("workspace_bytes", _size)]


# entry point -> its argument struct; size queries of the backward passes
ENTRIES = {"gdr2_conv_forward": ConvArgs, "gdr2_conv_step": ConvStepArgs, "gdr2_conv_backward": ConvBwdArgs,
           "gdr2_scan_forward": ScanArgs, "gdr2_scan_step": ScanStepArgs, "gdr2_scan_backward": ScanBwdArgs,
           "gdr2_norm_forward": NormArgs, "gdr2_norm_backward": NormBwdArgs}
SIZES = {"gdr2_conv_backward_workspace_size": ConvBwdArgs, "gdr2_scan_workspace_size": ScanArgs,
         "gdr2_scan_backward_workspace_size": ScanBwdArgs, "gdr2_norm_backward_workspace_size": NormBwdArgs}


# The single-token steps are all host time at small batches: their argument
# structs are packed in one go, and handed over as bytes.
_packed = {}
_CONV_STEP = struct.Struct("@3q4i5P")
_SCAN_STEP = struct.Struct("@10q4i14PNP")
assert _CONV_STEP.size == ctypes.sizeof(ConvStepArgs) and _SCAN_STEP.size == ctypes.sizeof(ScanStepArgs)


def _raw_stream(index: int) -> int:
    """The current stream of a device as a hipStream_t."""
    return torch._C._cuda_getCurrentRawStream(index)


def declare(lib):
    """Signatures of the layer operators in a loaded library."""
    for name, args in ENTRIES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = ctypes.c_int, [ctypes.POINTER(args), _vp]
        f = _packed[name] = lib[name]          # a second object of the same function
        f.restype, f.argtypes = ctypes.c_int, [ctypes.c_char_p, _vp]
    for name, args in SIZES.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = _size, [ctypes.POINTER(args)]
    lib.gdr2_scan_chunk_count.restype = _c_i64
    lib.gdr2_scan_chunk_count.argtypes = [_c_i64, _c_i64, ctypes.c_int]
    return lib


# ---- argument checks -------------------------------------------------------

def _row_stride(t: torch.Tensor, name: str, lead: int, width: int) -> int:
    """Elements between consecutive rows: the first ``lead`` dimensions number
    the rows, the others hold ``width`` dense elements."""
    if t.is_contiguous():
        return width
    if t.numel() == 0:
        return width
    shape, stride = t.shape, t.stride()
    step = 1
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] != 1:
            if stride[d] != step:
                raise ValueError(f"{name}: the elements of a row must be contiguous")
            step *= shape[d]
    ld = None
    for d in range(lead - 1, -1, -1):
        if shape[d] == 1:
            continue
        if ld is None:
            ld, span = stride[d], stride[d] * shape[d]
            if ld < width:              # an expanded dimension has stride 0
                raise ValueError(f"{name}: rows must not overlap")
        elif stride[d] != span:
            raise ValueError(f"{name}: rows must be equally spaced")
        else:
            span *= shape[d]
    return width if ld is None else ld


def _rows_dtype(t: torch.Tensor):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _mode(table, value, name: str) -> int:
    if value not in table:
        raise ValueError(f"unknown {name} {value!r} ({', '.join(map(repr, table))})")
    return table[value]


def _on(dev, dense, rows, names: str):
    """Every tensor on ``dev``, the ``dense`` ones contiguous; ``names``
    (dense first) only serve the message."""
    if dev.type == "cuda":
        for t in dense:
            if t is not None and (t.device != dev or not t.is_contiguous()):
                break
        else:
            for t in rows:
                if t is not None and t.device != dev:
                    break
            else:
                return
    for i, (n, t) in enumerate(zip(names.split(), (*dense, *rows))):
        if t is None:
            continue
        if i < len(dense):
            _req_dev(t, n, dev)
        elif not t.is_cuda:
            raise ValueError(f"{n} must be a device tensor")
        elif t.device != dev:
            raise ValueError(f"{n} is on {t.device}, expected {dev}")


def _offsets(offsets) -> int:
    """Number of sequences of a packed batch."""
    _req_shape(offsets, "offsets", torch.int64)
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError(f"offsets must have shape (B + 1,), got {tuple(offsets.shape)}")
    return offsets.shape[0] - 1


def _call(entry: str, args, dev):
    """Calls an entry point with its argument struct (a ctypes Structure, or
    the same bytes packed) on the current stream of ``dev``."""
    lib = load_library()
    f = _packed[entry] if type(args) is bytes else getattr(lib, entry)
    a = args if type(args) is bytes else ctypes.byref(args)
    index = dev.index
    if torch.cuda.current_device() == index:
        status = f(a, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = f(a, _raw_stream(index))
    if status:
        _check(lib, status)


def _with_workspace(size: str, args, workspace, dev):
    """Fills the workspace fields; the size depends on the device's compute
    units, so it is asked for with that device current."""
    f = getattr(load_library(), size)
    if torch.cuda.current_device() == dev.index:
        need = int(f(ctypes.byref(args)))
    else:
        with torch.cuda.device(dev):
            need = int(f(ctypes.byref(args)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None:
        args.workspace, args.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


def _empty(t, shape, like):
    return like.new_empty(shape) if t is None else t


def _grad_buffers(out, dev, **want):
    """The tensors gradients are written to, by name: the caller's ``out[name]``
    or fresh memory; ``want`` gives (dtype, shape), or None for no gradient."""
    out = out or {}
    for n in out:
        if want.get(n) is None:
            raise ValueError(f"out: no gradient {n!r} is formed ({', '.join(k for k, v in want.items() if v)})")
    g = {}
    for n, spec in want.items():
        if spec is not None and n in out:
            _req_shape(out[n], n, *spec)
            _req_dev(out[n], n, dev)
            g[n] = out[n]
        else:
            g[n] = None if spec is None else torch.empty(spec[1], dtype=spec[0], device=dev)
    return g


# ---- convolution -----------------------------------------------------------

def check_conv_shapes(x, weight, bias=None, state0=None, offsets=None):
    """Dtypes and shapes of the convolution's inputs; returns (B, T, C, K)."""
    _rows_dtype(x)
    if weight.dim() != 2:
        raise ValueError(f"weight must have shape (C, width), got {tuple(weight.shape)}")
    C, K = weight.shape
    _req_shape(weight, "weight", torch.float32)
    if offsets is None:
        if x.dim() != 3:
            raise ValueError(f"x must have shape (B, T, C), got {tuple(x.shape)}")
        B, T = x.shape[:2]
    else:
        if x.dim() != 2:
            raise ValueError(f"packed x must have shape (T, C), got {tuple(x.shape)}")
        T = x.shape[0]
        B = _offsets(offsets)
    _req_shape(x, "x", None, tuple(x.shape[:-1]) + (C,))
    if bias is not None:
        _req_shape(bias, "bias", torch.float32, (C,))
    if state0 is not None:
        _req_shape(state0, "state0", x.dtype, (B, K - 1, C))
    return B, T, C, K


def conv_forward(x, weight, bias=None, state0=None, offsets=None, activation="silu", out=None, state_out=None,
                 final_state: bool = True):
    """Short causal depthwise convolution.  x [B,T,C] (packed [T,C]); weight
    float32 [C,K], K in 2..4; bias float32 [C]; state0 [B,K-1,C], the rows
    before each sequence, oldest first (zero when None).  activation None or
    'silu'.  Returns (y, state): state [B,K-1,C] is the last K-1 inputs of
    each sequence, the state0 of its continuation (None when final_state is
    false and no state_out is given; state_out may be state0)."""
    B, T, C, K = check_conv_shapes(x, weight, bias, state0, offsets)
    act = _mode(ACTIVATIONS, activation, "activation")
    if out is not None:
        _req_shape(out, "out", x.dtype, tuple(x.shape))
    if state_out is not None:
        _req_shape(state_out, "state_out", x.dtype, (B, K - 1, C))
    ld = _row_stride(x, "x", x.dim() - 1, C)
    _on(x.device, (weight, bias, state0, offsets, out, state_out), (x,), "weight bias state0 offsets out state_out x")
    out = _empty(out, x.shape, x)
    if state_out is None and final_state:
        state_out = x.new_empty((B, max(K - 1, 0), C))
    a = ConvArgs(B, T, C, ld, K, _dtype_code(x), act, 0, x.data_ptr(), weight.data_ptr(), _ptr(bias),
                 _ptr(state0), _ptr(offsets), out.data_ptr(), _ptr(state_out))
    _call("gdr2_conv_forward", a, x.device)
    return out, state_out


def conv_step(state, x, weight, bias=None, activation="silu", out=None):
    """The convolution for one token of each of N sequences, in place on
    ``state`` [N,K-1,C]; x [N,C].  Returns y [N,C]."""
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"x and weight must have shapes (N, C) and (C, width), got {tuple(x.shape)} and "
                         f"{tuple(weight.shape)}")
    act = _mode(ACTIVATIONS, activation, "activation")
    (C, K), N, e = weight.shape, x.shape[0], x.dtype
    if not (x.shape == (N, C) and state.shape == (N, K - 1, C) and (e is torch.bfloat16 or e is torch.float32)
            and state.dtype is e and weight.dtype is torch.float32
            and (bias is None or bias.dtype is torch.float32 and bias.shape == (C,))):
        _rows_dtype(x)
        _req_shape(x, "x", None, (N, C))
        _req_shape(weight, "weight", torch.float32)
        _req_shape(state, "state", e, (N, K - 1, C))
        _req_shape(bias, "bias", torch.float32, (C,))
    if out is not None:
        _req_shape(out, "out", x.dtype, (N, C))
    ld = _row_stride(x, "x", 1, C)
    dev = x.device
    _on(dev, (state, weight, bias, out), (x,), "state weight bias out x")
    out = _empty(out, (N, C), x)
    _call("gdr2_conv_step", _CONV_STEP.pack(N, C, ld, K, _dtype_code(x), act, 0, state.data_ptr(), x.data_ptr(),
                                            weight.data_ptr(), 0 if bias is None else bias.data_ptr(), out.data_ptr()), dev)
    return out


def conv_backward(x, weight, dy, bias=None, state0=None, offsets=None, activation="silu", dstate=None,
                  want_dstate0=None, out=None, workspace=None):
    """Gradients of ``conv_forward`` for dL/dy (shaped like y) and optionally
    dL/dstate ``dstate`` [B,K-1,C].  Returns a dict: dx, dweight, dbias (None
    without bias), dstate0 (by default when state0 is given); ``out``: a dict
    of tensors to write some of them into."""
    B, T, C, K = check_conv_shapes(x, weight, bias, state0, offsets)
    act = _mode(ACTIVATIONS, activation, "activation")
    _req_shape(dy, "dy", x.dtype, tuple(x.shape))
    if dstate is not None:
        _req_shape(dstate, "dstate", x.dtype, (B, K - 1, C))
    ld = _row_stride(x, "x", x.dim() - 1, C)
    dev = x.device
    _on(dev, (weight, bias, state0, offsets, dy, dstate, workspace), (x,),
        "weight bias state0 offsets dy dstate workspace x")
    want = state0 is not None if want_dstate0 is None else want_dstate0
    e, f32 = x.dtype, torch.float32
    g = _grad_buffers(out, dev, dx=(e, tuple(x.shape)), dweight=(f32, (C, K)), dbias=None if bias is None else (f32, (C,)),
                      dstate0=(e, (B, max(K - 1, 0), C)) if want else None)
    a = ConvBwdArgs(B, T, C, ld, K, _dtype_code(x), act, 0, x.data_ptr(), weight.data_ptr(), _ptr(bias),
                    _ptr(state0), _ptr(offsets), dy.data_ptr(), _ptr(dstate), g["dx"].data_ptr(), g["dweight"].data_ptr(),
                    _ptr(g["dbias"]), _ptr(g["dstate0"]))
    workspace = _with_workspace("gdr2_conv_backward_workspace_size", a, workspace, dev)
    _call("gdr2_conv_backward", a, dev)
    return g


# ---- scan ------------------------------------------------------------------

def check_scan_shapes(x, dt, A, Bt, Ct, skip=None, z=None, dt_bias=None, offsets=None, lead=None):
    """Dtypes and shapes of the scan's inputs; returns (B, T, C, N, G).
    ``lead``: the number of leading dimensions (a step has one)."""
    if lead == 1 and A.dim() == 2 and Bt.dim() == 3:      # a step: all in one expression, the reasons below
        (B, _), (C, N), G, e = x.shape[:2] if x.dim() == 2 else (0, 0), A.shape, Bt.shape[1], x.dtype
        if (x.shape == (B, C) == dt.shape and Bt.shape == (B, G, N) == Ct.shape and A.dtype is torch.float32
                and (e is torch.bfloat16 or e is torch.float32) and dt.dtype is e and Bt.dtype is e and Ct.dtype is e
                and (z is None or z.dtype is e and z.shape == (B, C))
                and (skip is None or skip.dtype is torch.float32 and skip.shape == (C,))
                and (dt_bias is None or dt_bias.dtype is torch.float32 and dt_bias.shape == (C,))):
            return B, 1, C, N, G
    _rows_dtype(x)
    if A.dim() != 2:
        raise ValueError(f"A must have shape (C, N), got {tuple(A.shape)}")
    _req_shape(A, "A", torch.float32)
    C, N = A.shape
    nlead = lead if lead is not None else 2 if offsets is None else 1
    if x.dim() != nlead + 1:
        raise ValueError(f"x must have {nlead + 1} dimensions, got shape {tuple(x.shape)}")
    rows = tuple(x.shape[:-1])
    _req_shape(x, "x", None, rows + (C,))
    _req_shape(dt, "dt", x.dtype, rows + (C,))
    if Bt.dim() != nlead + 2:
        raise ValueError(f"Bt must have shape {rows + ('G', N)}, got {tuple(Bt.shape)}")
    G = Bt.shape[-2]
    _req_shape(Bt, "Bt", x.dtype, rows + (G, N))
    _req_shape(Ct, "Ct", x.dtype, rows + (G, N))
    if z is not None:
        _req_shape(z, "z", x.dtype, rows + (C,))
    for n, t in (("skip", skip), ("dt_bias", dt_bias)):
        if t is not None:
            _req_shape(t, n, torch.float32, (C,))
    if offsets is not None:
        return _offsets(offsets), rows[0], C, N, G
    return rows[0], rows[1] if nlead == 2 else 1, C, N, G


def scan_args(B, T, C, N, G, x, dt, A, Bt, Ct, skip, z, dt_bias, softplus, offsets=None, algo="auto") -> ScanArgs:
    lead = x.dim() - 1
    return ScanArgs(B, T, C, N, G, _row_stride(x, "x", lead, C), _row_stride(dt, "dt", lead, C),
                    _row_stride(Bt, "Bt", lead, G * N), _row_stride(Ct, "Ct", lead, G * N),
                    0 if z is None else _row_stride(z, "z", lead, C), _dtype_code(x),
                    SCAN_SOFTPLUS if softplus else 0, _mode(SCAN_ALGOS, algo, "algo"), 0, x.data_ptr(), dt.data_ptr(), Bt.data_ptr(),
                    Ct.data_ptr(), _ptr(z), A.data_ptr(), _ptr(skip), _ptr(dt_bias), None, _ptr(offsets))


def scan_chunk_count(B: int, T: int, packed: bool = False) -> int:
    """Rows of h_chunks for B sequences of T tokens (packed: T rows in all)."""
    return int(load_library().gdr2_scan_chunk_count(B, T, int(packed)))


def scan_forward(x, dt, A, Bt, Ct, skip=None, z=None, dt_bias=None, h0=None, offsets=None, softplus: bool = True,
                 out=None, h_out=None, final_state: bool = True, chunk_states=None, algo: str = "auto", workspace=None):
    """Selective state space scan.  x, dt, z [B,T,C]; Bt, Ct [B,T,G,N] (packed
    without B); A float32 [C,N]; skip, dt_bias float32 [C]; h0 float32 [B,C,N].
    Returns (y, h) or, when chunk_states is True or a float32 tensor
    [scan_chunk_count,C,N], (y, h, h_chunks): the state before every 32nd
    token, which ``scan_backward`` takes.  h is the state after each sequence
    (None when final_state is false and no h_out is given; h_out may be h0).
    Tokens masked with dt = -inf (or the dtype's lowest value) leave the state
    as it is, with softplus."""
    B, T, C, N, G = check_scan_shapes(x, dt, A, Bt, Ct, skip, z, dt_bias, offsets)
    for n, t in (("h0", h0), ("h_out", h_out)):
        if t is not None:
            _req_shape(t, n, torch.float32, (B, C, N))
    if out is not None:
        _req_shape(out, "out", x.dtype, tuple(x.shape))
    ck = chunk_states if isinstance(chunk_states, torch.Tensor) else None
    if ck is not None:
        _req_shape(ck, "chunk_states", torch.float32, (scan_chunk_count(B, T, offsets is not None), C, N))
    dev = x.device
    _on(dev, (A, skip, dt_bias, h0, offsets, out, h_out, ck, workspace), (x, dt, Bt, Ct, z),
        "A skip dt_bias h0 offsets out h_out chunk_states workspace x dt Bt Ct z")
    a = scan_args(B, T, C, N, G, x, dt, A, Bt, Ct, skip, z, dt_bias, softplus, offsets, algo)
    out = _empty(out, x.shape, x)
    if h_out is None and final_state:
        h_out = A.new_empty((B, C, N))
    if ck is None and chunk_states:
        ck = A.new_empty((scan_chunk_count(B, T, offsets is not None), C, N))
    a.h0, a.y, a.h_out, a.h_chunks = _ptr(h0), out.data_ptr(), _ptr(h_out), _ptr(ck)
    workspace = _with_workspace("gdr2_scan_workspace_size", a, workspace, dev)
    _call("gdr2_scan_forward", a, dev)
    return (out, h_out) if ck is None else (out, h_out, ck)


def scan_step(state, x, dt, A, Bt, Ct, skip=None, z=None, dt_bias=None, softplus: bool = True, out=None):
    """The scan for one token of each of B sequences, in place on ``state``
    float32 [B,C,N]; x, dt, z [B,C]; Bt, Ct [B,G,N].  Returns y [B,C]."""
    B, _, C, N, G = check_scan_shapes(x, dt, A, Bt, Ct, skip, z, dt_bias, None, lead=1)
    _req_shape(state, "state", torch.float32, (B, C, N))
    if out is not None:
        _req_shape(out, "out", x.dtype, (B, C))
    dev = x.device
    _on(dev, (state, A, skip, dt_bias, out), (x, dt, Bt, Ct, z), "state A skip dt_bias out x dt Bt Ct z")
    out = _empty(out, (B, C), x)
    _call("gdr2_scan_step", _SCAN_STEP.pack(
        B, 1, C, N, G, _row_stride(x, "x", 1, C), _row_stride(dt, "dt", 1, C), _row_stride(Bt, "Bt", 1, G * N),
        _row_stride(Ct, "Ct", 1, G * N), 0 if z is None else _row_stride(z, "z", 1, C), _dtype_code(x),
        SCAN_SOFTPLUS if softplus else 0, 0, 0, x.data_ptr(), dt.data_ptr(), Bt.data_ptr(), Ct.data_ptr(),
        0 if z is None else z.data_ptr(), A.data_ptr(), 0 if skip is None else skip.data_ptr(),
        0 if dt_bias is None else dt_bias.data_ptr(), 0, 0, out.data_ptr(), 0, 0, 0, 0, state.data_ptr()), dev)
    return out


def scan_backward(x, dt, A, Bt, Ct, dy, h_chunks, skip=None, z=None, dt_bias=None, offsets=None, softplus: bool = True,
                  dh_out=None, want_dh0: bool = True, algo: str = "auto", out=None, workspace=None):
    """Gradients of ``scan_forward`` for dL/dy and optionally dL/dh ``dh_out``
    float32 [B,C,N]; h_chunks as the forward of the same inputs returned them.
    Returns a dict: dx, ddt, dBt, dCt, dz (None without z) in the rows' dtype;
    dA, dskip, ddt_bias (None without their parameter), dh0 float32; ``out``:
    a dict of tensors to write some of them into (dh0 may be dh_out)."""
    B, T, C, N, G = check_scan_shapes(x, dt, A, Bt, Ct, skip, z, dt_bias, offsets)
    _req_shape(dy, "dy", x.dtype, tuple(x.shape))
    _req_shape(h_chunks, "h_chunks", torch.float32, (scan_chunk_count(B, T, offsets is not None), C, N))
    if dh_out is not None:
        _req_shape(dh_out, "dh_out", torch.float32, (B, C, N))
    dev = x.device
    _on(dev, (A, skip, dt_bias, offsets, dy, h_chunks, dh_out, workspace), (x, dt, Bt, Ct, z),
        "A skip dt_bias offsets dy h_chunks dh_out workspace x dt Bt Ct z")
    f = scan_args(B, T, C, N, G, x, dt, A, Bt, Ct, skip, z, dt_bias, softplus, offsets, algo)
    f.h_chunks = h_chunks.data_ptr()

    def like(t):
        return None if t is None else (t.dtype, tuple(t.shape))

    g = _grad_buffers(out, dev, dx=like(x), ddt=like(dt), dBt=like(Bt), dCt=like(Ct), dz=like(z), dA=like(A), dskip=like(skip),
                      ddt_bias=like(dt_bias), dh0=(torch.float32, (B, C, N)) if want_dh0 else None)
    a = ScanBwdArgs(f, dy.data_ptr(), _ptr(dh_out), *(_ptr(g[n]) for n in ("dx", "ddt", "dBt", "dCt", "dz", "dA", "dskip",
                                                                          "ddt_bias", "dh0")))
    workspace = _with_workspace("gdr2_scan_backward_workspace_size", a, workspace, dev)
    _call("gdr2_scan_backward", a, dev)
    return g


# ---- norm ------------------------------------------------------------------

def check_norm_shapes(x, weight=None, bias=None, z=None):
    """Dtypes and shapes of the norm's inputs; returns (R, C)."""
    _rows_dtype(x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have shape (..., C), got {tuple(x.shape)}")
    C = x.shape[-1]
    for n, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _req_shape(t, n, torch.float32, (C,))
    if z is not None:
        _req_shape(z, "z", x.dtype, tuple(x.shape))
    return x.numel() // C, C


def norm_args(R, C, x, weight, bias, z, eps, kind) -> NormArgs:
    lead = x.dim() - 1
    return NormArgs(R, C, _row_stride(x, "x", lead, C), 0 if z is None else _row_stride(z, "z", lead, C), _dtype_code(x),
                    _mode(KINDS, kind, "kind"), eps, 0, x.data_ptr(), _ptr(z), _ptr(weight), _ptr(bias))


def norm_forward(x, weight=None, bias=None, z=None, eps: float = 1e-5, kind: str = "layer", out=None):
    """Norm of the last dimension: kind 'layer' (mean taken off) or 'rms';
    weight, bias float32 [C]; with a gate z (shaped like x) the result is
    multiplied by silu(z)."""
    R, C = check_norm_shapes(x, weight, bias, z)
    if out is not None:
        _req_shape(out, "out", x.dtype, tuple(x.shape))
    _on(x.device, (weight, bias, out), (x, z), "weight bias out x z")
    a = norm_args(R, C, x, weight, bias, z, eps, kind)
    out = _empty(out, x.shape, x)
    a.y = out.data_ptr()
    _call("gdr2_norm_forward", a, x.device)
    return out


def norm_backward(x, dy, weight=None, bias=None, z=None, eps: float = 1e-5, kind: str = "layer", out=None, workspace=None):
    """Gradients of ``norm_forward`` for dL/dy.  Returns a dict: dx, dz (None
    without z), dweight and dbias (float32, None without their parameter);
    ``out``: a dict of tensors to write some of them into."""
    R, C = check_norm_shapes(x, weight, bias, z)
    _req_shape(dy, "dy", x.dtype, tuple(x.shape))
    dev = x.device
    _on(dev, (weight, bias, dy, workspace), (x, z), "weight bias dy workspace x z")
    f = norm_args(R, C, x, weight, bias, z, eps, kind)
    rows, param = (x.dtype, tuple(x.shape)), (torch.float32, (C,))
    g = _grad_buffers(out, dev, dx=rows, dz=None if z is None else rows, dweight=None if weight is None else param,
                      dbias=None if bias is None else param)
    a = NormBwdArgs(f, dy.data_ptr(), g["dx"].data_ptr(), _ptr(g["dz"]), _ptr(g["dweight"]), _ptr(g["dbias"]))
    workspace = _with_workspace("gdr2_norm_backward_workspace_size", a, workspace, dev)
    _call("gdr2_norm_backward", a, dev)
    return g
