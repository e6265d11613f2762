"""Host-side tests of the block operators' C ABI and binding (no GPU needed):
every invalid or unsupported argument is refused before any launch.  As in
tests/test_boundary_host.py the pointers are fake, aligned, far apart, and
never dereferenced on these paths."""
import ctypes

import pytest
import torch

from gated_delta_rule_86_amd import block, gdr2
from tests.test_boundary_host import _gpu_visible, fake, lib  # noqa: F401
from tests.test_layer_host import _get, _point, _set

pytestmark = pytest.mark.skipif(_gpu_visible(), reason="host-only tests use fake device pointers")

INV, UNS, WSP = gdr2.ERR_INVALID_ARG, gdr2.ERR_UNSUPPORTED, gdr2.ERR_WORKSPACE


def pack():
    a = block.PackArgs(R=70, C=64, x_stride=80, dtype=gdr2.BF16)
    _point(a)
    return a


def unpack():
    a = block.UnpackArgs(R=70, C=64, dtype=gdr2.BF16)
    _point(a)
    return a


def add_norm():
    a = block.AddNormArgs(R=70, C=64, x_stride=64, res_stride=80, dtype=gdr2.BF16, res_dtype=gdr2.F32, kind=1, eps=1e-5)
    _point(a)
    return a


def add_norm_bwd():
    a = block.AddNormBwdArgs(R=70, C=64, dtype=gdr2.BF16, res_dtype=gdr2.F32, kind=0, eps=1e-5)
    _point(a, skip=("codes", "scales"))
    a.workspace_bytes = 1 << 30
    return a


def add_norm_bwd8():
    a = add_norm_bwd()
    a.h = None
    a.h8.codes, a.h8.scales = fake(40), fake(41)
    return a


def _glr(T=6400):
    return block.GlrArgs(B=2, T=T, C=64, x_stride=64, r_stride=128, i_stride=128, dtype=gdr2.BF16, algo=gdr2.ALGOS["segmented"])


def glr():
    a = _glr()
    _point(a, skip=("offsets",))
    a.workspace_bytes = 1 << 30
    return a


def glr_step():
    a = block.GlrStepArgs(N=5, C=64, x_stride=64, r_stride=128, i_stride=128, dtype=gdr2.BF16)
    _point(a)
    return a


def glr_bwd():
    a = block.GlrBwdArgs(f=_glr())
    _point(a, skip=("offsets", "codes", "scales"))
    a.workspace_bytes = 1 << 30
    return a


def glr_bwd8():
    a = block.GlrBwdArgs(f=_glr())
    _point(a, skip=("offsets", "x", "r", "i"))
    a.f.x_stride = a.f.r_stride = a.f.i_stride = 0
    a.workspace_bytes = 1 << 30
    return a


MAKE = {"pack": ("gdr2_pack_rows", pack), "unpack": ("gdr2_unpack_rows", unpack), "add_norm": ("gdr2_add_norm_forward", add_norm),
        "add_norm_bwd": ("gdr2_add_norm_backward", add_norm_bwd), "add_norm_bwd8": ("gdr2_add_norm_backward", add_norm_bwd8),
        "glr": ("gdr2_glr_forward", glr), "glr_step": ("gdr2_glr_step", glr_step), "glr_bwd": ("gdr2_glr_backward", glr_bwd),
        "glr_bwd8": ("gdr2_glr_backward", glr_bwd8)}

CASES = {
    "pack": [("R", -1, INV), ("C", 0, INV), ("x_stride", 63, INV), ("dtype", 2, INV), ("reserved", 1, INV), ("R", 1 << 40, UNS),
             ("x_stride", 1 << 41, UNS)],
    "unpack": [("R", -1, INV), ("C", -1, INV), ("C", 1 << 25, UNS), ("dtype", -1, INV), ("reserved", 1, INV), ("R", 1 << 40, UNS)],
    "add_norm": [("R", -1, INV), ("C", 0, INV), ("x_stride", 63, INV), ("res_stride", 63, INV), ("dtype", 2, INV), ("res_dtype", 3, INV),
                 ("kind", 2, INV), ("eps", -1.0, INV), ("eps", float("inf"), INV),
                 ("eps", float("nan"), INV), ("R", 1 << 40, UNS), ("residual", None, INV)],
    "add_norm_bwd": [("R", -1, INV), ("C", 0, INV), ("C", 16385, UNS), ("dtype", 2, INV), ("res_dtype", -1, INV), ("kind", -1, INV),
                     ("eps", float("nan"), INV), ("workspace_bytes", 0, WSP), ("workspace", None, WSP), ("h8.codes", fake(60), INV)],
    "add_norm_bwd8": [("h", fake(60), INV), ("h8.codes", None, INV), ("h8.scales", None, INV)],
    "glr": [("B", -1, INV), ("T", -1, INV), ("C", 0, INV), ("x_stride", 63, INV), ("r_stride", 63, INV), ("i_stride", 0, INV),
            ("x_stride", (1 << 22) + 1, UNS), ("dtype", 2, INV), ("algo", 3, INV), ("T", 1 << 41, UNS), ("B", 1 << 33, UNS),
            ("workspace_bytes", 16, WSP), ("workspace", None, WSP)],
    "glr_step": [("N", -1, INV), ("C", 0, INV), ("x_stride", 63, INV), ("r_stride", 63, INV), ("i_stride", 63, INV), ("dtype", 7, INV),
                 ("reserved", 1, INV), ("N", 1 << 40, UNS)],
    "glr_bwd": [("f.B", -1, INV), ("f.C", 0, INV), ("f.algo", 9, INV), ("f.r_stride", 63, INV), ("f.x", None, INV), ("f.r", None, INV),
                ("f.x8.codes", fake(60), INV), ("workspace_bytes", 16, WSP)],
    "glr_bwd8": [("f.x", fake(60), INV), ("f.x8.codes", None, INV), ("f.r8.scales", None, INV), ("f.i8.codes", None, INV),
                 ("workspace", None, WSP)],
}
# buffers a call can do without, and those it does not read
OPTIONAL = {"residual", "weight", "bias", "h", "y", "y8.codes", "h8.codes", "y8.scales", "h8.scales", "dh", "dresidual", "dx", "dweight",
            "dbias", "h0", "h_out", "h_chunks", "dh_out", "dh0", "workspace", "x8.codes", "x8.scales", "r8.codes", "r8.scales",
            "i8.codes", "i8.scales"}
IGNORED = {"f.h0", "f.y", "f.h_out", "f.workspace"}
OUTPUTS = {"y", "h", "h_out", "h_chunks", "state", "dx", "dr", "di", "dA", "dh0", "dresidual", "dweight", "dbias", "workspace",
           "codes", "scales"}
INPUTS = {"unpack": {"rows.codes", "rows.scales"}, "add_norm_bwd": {"h"}, "add_norm_bwd8": {"h8.codes", "h8.scales"},
          "glr_bwd": {"f.h_chunks"},
          "glr_bwd8": {"f.h_chunks", *(f"f.{n}8.{p}" for n in "xri" for p in ("codes", "scales"))}}
ALIAS = {("h_out", "h0"), ("dh0", "dh_out"), ("dresidual", "dh")}


def call(lib, kind, a):  # noqa: F811
    return getattr(lib, MAKE[kind][0])(ctypes.byref(a), None)


@pytest.mark.parametrize("kind,field,value,status", [(n, *c) for n, cs in CASES.items() for c in cs])
def test_refuses_sizes_and_modes(lib, kind, field, value, status):  # noqa: F811
    a = MAKE[kind][1]()
    _set(a, field, value)
    assert call(lib, kind, a) == status, lib.gdr2_last_error()
    assert lib.gdr2_last_error()


def test_refuses_bf16_streams_of_fp32_rows(lib):  # noqa: F811
    for kind in ("add_norm", "add_norm_bwd"):
        a = MAKE[kind][1]()
        a.dtype, a.res_dtype = gdr2.F32, gdr2.BF16
        assert call(lib, kind, a) == UNS


@pytest.mark.parametrize("kind", list(MAKE))
def test_refuses_null_args(lib, kind):  # noqa: F811
    assert getattr(lib, MAKE[kind][0])(None, None) == INV


def _pointers(kind):
    a = MAKE[kind][1]()
    names = [p for p in _point(type(a)()) if _get(a, p) is not None]
    return [p for p in names if p not in IGNORED]


@pytest.mark.parametrize("kind", list(MAKE))
def test_refuses_missing_pointers(lib, kind):  # noqa: F811
    required = {"add_norm_bwd": {"h"}, "glr_bwd": {"f.h_chunks"}, "glr_step": {"y"}, "unpack": {"y"}, "glr": {"y"},
                "glr_bwd8": INPUTS["glr_bwd8"], "add_norm_bwd8": INPUTS["add_norm_bwd8"]}.get(kind, set())
    both = {"dx", "dresidual"} if kind.startswith("add_norm") else set()
    checked = 0
    for p in _pointers(kind):
        last = p.removeprefix("f.")
        if (last in OPTIONAL and p not in required and not (kind.startswith("glr_bwd") and last == "dx")) or last in both:
            continue
        a = MAKE[kind][1]()
        _set(a, p, None)
        assert call(lib, kind, a) == INV, p
        assert p.split(".")[-1].encode() in lib.gdr2_last_error() or b"both given" in lib.gdr2_last_error(), (p, lib.gdr2_last_error())
        checked += 1
    assert checked


def test_refuses_half_of_an_output(lib):  # noqa: F811
    """Codes without their scales, one of three checkpoints, no output at all."""
    for kind, names in (("add_norm", ("y8", "h8")), ("glr", ("x8", "r8", "i8"))):
        for n in names:
            for part in ("codes", "scales"):
                a = MAKE[kind][1]()
                _set(a, f"{n}.{part}", None)
                assert call(lib, kind, a) == INV and f"{n}.{part} is NULL".encode() in lib.gdr2_last_error()
    a = glr()
    a.r8.codes = a.r8.scales = None
    assert call(lib, "glr", a) == INV
    a = add_norm()
    for n in ("h", "y", "y8.codes", "y8.scales", "h8.codes", "h8.scales"):
        _set(a, n, None)
    assert call(lib, "add_norm", a) == INV and b"no output" in lib.gdr2_last_error()
    a = add_norm_bwd()
    a.dx = a.dresidual = None
    assert call(lib, "add_norm_bwd", a) == INV and b"no output" in lib.gdr2_last_error()


@pytest.mark.parametrize("kind", list(MAKE))
def test_refuses_misaligned_and_overlapping(lib, kind):  # noqa: F811
    ptrs = _pointers(kind)
    rows = {"x", "r", "i", "residual"}
    for p in ptrs:
        a = MAKE[kind][1]()
        _set(a, p, _get(a, p) + (1 if p.split(".")[-1] in rows else 8))
        assert call(lib, kind, a) == INV and b"aligned" in lib.gdr2_last_error(), p
    pairs = 0
    for p in ptrs:
        if p.split(".")[-1] not in OUTPUTS or p in INPUTS.get(kind, ()):
            continue
        for o in ptrs:
            if o == p:
                continue
            for shift in (0, 16):
                if (p.removeprefix("f."), o) in ALIAS and shift == 0:
                    continue
                a = MAKE[kind][1]()
                # the other buffer starts `shift` bytes into this one
                _set(a, o, _get(a, p) + shift)
                assert call(lib, kind, a) == INV and b"overlaps" in lib.gdr2_last_error(), (p, o, shift, lib.gdr2_last_error())
                pairs += 1
    assert pairs


def test_in_place(lib):  # noqa: F811
    """The pairs that may be one buffer pass the overlap rule (a buffer that is
    missing on purpose is what is refused, and it is asked for before)."""
    a = add_norm()
    a.res_stride, a.h = 64, a.residual
    a.x = a.y8.codes                                       # .. and this is what overlaps
    assert call(lib, "add_norm", a) == INV and b"y8.codes overlaps x" in lib.gdr2_last_error()
    a = add_norm()
    a.h = a.residual                                       # rows 80 elements apart are no dense stream
    assert call(lib, "add_norm", a) == INV and b"h overlaps residual" in lib.gdr2_last_error()
    for kind, out, other in (("glr", "h_out", "h0"), ("glr_bwd", "dh0", "dh_out"), ("add_norm_bwd", "dresidual", "dh")):
        a = MAKE[kind][1]()
        _set(a, out, _get(a, other))
        _set(a, "y" if kind == "glr" else "dx", a.workspace)
        assert call(lib, kind, a) == INV and b"workspace" in lib.gdr2_last_error(), lib.gdr2_last_error()


def test_empty_batches_launch_nothing(lib):  # noqa: F811
    for kind, field in (("pack", "R"), ("unpack", "R"), ("add_norm", "R"), ("glr", "B"), ("glr_step", "N")):
        a = MAKE[kind][1]()
        _set(a, field, 0)
        assert call(lib, kind, a) == gdr2.OK, (kind, lib.gdr2_last_error())


def test_workspace_sizes(lib):  # noqa: F811
    for kind, size in (("add_norm_bwd", "gdr2_add_norm_backward_workspace_size"), ("glr", "gdr2_glr_workspace_size"),
                       ("glr_bwd", "gdr2_glr_backward_workspace_size"), ("glr_bwd8", "gdr2_glr_backward_workspace_size")):
        a = MAKE[kind][1]()
        need = getattr(lib, size)(ctypes.byref(a))
        assert need > 0
        a.workspace_bytes = need - 1
        assert call(lib, kind, a) == WSP
        assert getattr(lib, size)(None) == 0
    a = glr()
    a.algo = gdr2.ALGOS["staged"]
    assert lib.gdr2_glr_workspace_size(ctypes.byref(a)) == 0          # one pass
    b = add_norm_bwd()
    b.dweight = b.dbias = None
    assert lib.gdr2_add_norm_backward_workspace_size(ctypes.byref(b)) == 0
    assert [lib.gdr2_glr_chunk_count(*v) for v in ((2, 100, 0), (2, 64, 0), (3, 100, 1), (0, 9, 1), (2, 0, 0), (2, 0, 1))] \
        == [14, 8, 9, 0, 0, 2]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,C,ok", [((1 << 22) - 1, 64, True), (1 << 23, 64, False), (1 << 23, 1, False), ((1 << 22) - 1, 1, True),
                                    (1 << 20, 2048, False)])
def test_refuses_more_workgroups_than_one_launch_takes(lib, B, C, ok, backward):  # noqa: F811
    """A workgroup of 512 threads counts twice; every pointer is NULL, so nothing launches."""
    f = block.GlrArgs(B=B, T=1, C=C, x_stride=C, r_stride=C, i_stride=C, dtype=gdr2.F32)
    a = block.GlrBwdArgs(f=f) if backward else f
    status = getattr(lib, "gdr2_glr_backward" if backward else "gdr2_glr_forward")(ctypes.byref(a), None)
    assert status == UNS if not ok else status in (INV, WSP), lib.gdr2_last_error()


# ---- the binding's own checks (before any device is touched) ---------------

def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _r8(*shape, scales=None):
    return block.Rows8(_t(*shape, dtype=block.CODES), _t(*(scales or (*shape[:-1], -(-shape[-1] // 32))), dtype=torch.uint8).view(block.SCALES))


def test_binding_refuses_rows8():
    x = _t(3, 40)
    for f in (lambda: block.pack_rows(_t(3, 0)), lambda: block.pack_rows(x.t()), lambda: block.pack_rows(x, out=_r8(3, 41)),
              lambda: block.pack_rows(x, out=_r8(3, 40, scales=(3, 1))), lambda: block.unpack_rows(x), lambda: block.unpack_rows(_r8(3, 40, scales=(3, 3))),
              lambda: block.unpack_rows(_r8(3, 40), torch.float32, out=_t(3, 41)), lambda: block.unpack_rows((x,))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: block.pack_rows(x.half()), lambda: block.pack_rows(x, out=(x, x)), lambda: block.pack_rows(x, out=x),
              lambda: block.unpack_rows(_r8(3, 40), torch.float16), lambda: block.unpack_rows((x, x))):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: block.pack_rows(x), lambda: block.unpack_rows(_r8(3, 40))):
        with pytest.raises(ValueError, match="device tensor"):
            f()


def test_binding_refuses_add_norm():
    x = _t(3, 4, 8)
    for kw in (dict(residual=_t(12, 8)), dict(weight=_t(7)), dict(bias=_t(9)), dict(kind="batch"), dict(want=("h", "z")),
               dict(out={"z": x}), dict(want=("y",), out={"h": x}), dict(out={"h": _t(3, 4, 9)}),
               dict(want=("y8",), out={"y8": _r8(3, 4, 9)}), dict(residual=_t(4, 3, 8).transpose(0, 1))):
        with pytest.raises(ValueError):
            block.add_norm_forward(x, **kw)
    with pytest.raises(ValueError):
        block.add_norm_forward(_t(3, 0))
    b = x.bfloat16()
    for f in (lambda: block.add_norm_forward(x, b), lambda: block.add_norm_forward(b, x.half()), lambda: block.add_norm_forward(x.half()),
              lambda: block.add_norm_forward(b, x, out={"h": b}), lambda: block.add_norm_forward(x, weight=_t(8, dtype=torch.bfloat16)),
              lambda: block.add_norm_backward(b, x), lambda: block.add_norm_backward(x, x, b),
              lambda: block.add_norm_backward(x, x, residual_dtype=torch.bfloat16), lambda: block.add_norm_backward(x.half(), x),
              lambda: block.add_norm_backward(_r8(3, 4, 8), x, residual_dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: block.add_norm_backward(_t(3, 4, 9), x), lambda: block.add_norm_backward(x, x, _t(3, 8)),
              lambda: block.add_norm_backward(_r8(3, 4, 9), x), lambda: block.add_norm_backward(x, x, weight=_t(9)),
              lambda: block.add_norm_backward(x, x, kind="z")):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError, match="device tensor"):
        block.add_norm_forward(x, x)
    with pytest.raises(ValueError, match="device tensor"):
        block.add_norm_backward(x, x)


def test_binding_refuses_glr():
    def good():
        return dict(x=_t(2, 5, 6), r=_t(2, 5, 6), i=_t(2, 5, 6), A=_t(6))
    offs = torch.zeros(3, dtype=torch.int64)
    for kw in (dict(r=_t(2, 5, 5)), dict(i=_t(2, 4, 6)), dict(A=_t(5)), dict(A=_t(6, 1)), dict(x=_t(10, 6)), dict(h0=_t(2, 5)),
               dict(h_out=_t(1, 6)), dict(out=_t(2, 5, 1)), dict(chunk_states=_t(3, 6)), dict(offsets=offs), dict(algo="fused"),
               dict(checkpoint=(_r8(2, 5, 6),)), dict(checkpoint=(_r8(2, 5, 6), _r8(2, 5, 6), _r8(2, 5, 7)))):
        with pytest.raises(ValueError):
            block.glr_forward(**{**good(), **kw})
    for kw in (dict(r=_t(2, 5, 6, dtype=torch.bfloat16)), dict(A=_t(6, dtype=torch.float64)), dict(x=_r8(2, 5, 6)),
               dict(x=_r8(2, 5, 6), r=_r8(2, 5, 6), i=_r8(2, 5, 6)), dict(h0=_t(2, 6, dtype=torch.bfloat16))):
        with pytest.raises(TypeError):
            block.glr_forward(**{**good(), **kw})
    for kw in (dict(dy=_t(2, 5, 5)), dict(h_chunks=_t(3, 6)), dict(dh_out=_t(2, 5))):
        with pytest.raises(ValueError):
            block.glr_backward(**good(), **{"dy": _t(2, 5, 6), "h_chunks": _t(2, 6), **kw})
    with pytest.raises(TypeError):
        block.glr_backward(**good(), dy=_t(2, 5, 6, dtype=torch.bfloat16), h_chunks=_t(2, 6))
    for f in (lambda: block.glr_step(_t(2, 5), _t(2, 6), _t(2, 6), _t(2, 6), _t(6)),
              lambda: block.glr_step(_t(2, 6), _t(2, 6), _t(2, 6), _t(2, 6), _t(5)), lambda: block.glr_step(_t(2, 6), _t(1, 2, 6), _t(2, 6), _t(2, 6), _t(6))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError, match="device tensor"):
        block.glr_forward(**good())
    with pytest.raises(ValueError, match="device tensor"):
        block.glr_step(_t(2, 6), _t(2, 6), _t(2, 6), _t(2, 6), _t(6))
    with pytest.raises(ValueError, match="device tensor"):
        block.glr_backward(*(_r8(2, 5, 6) for _ in range(3)), _t(6), _t(2, 5, 6), _t(2, 6))
