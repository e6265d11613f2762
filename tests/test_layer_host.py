"""Host-side tests of the layer operators' C ABI and binding (no GPU needed):
every invalid or unsupported argument is refused before any launch.  As in
tests/test_boundary_host.py the pointers are fake, aligned, far apart, and
never dereferenced on these paths."""
import ctypes

import pytest
import torch

from gated_delta_rule_86_amd import gdr2, layer
from tests.test_boundary_host import _gpu_visible, fake, lib  # noqa: F401

pytestmark = pytest.mark.skipif(_gpu_visible(), reason="host-only tests use fake device pointers")

INV, UNS, WSP = gdr2.ERR_INVALID_ARG, gdr2.ERR_UNSUPPORTED, gdr2.ERR_WORKSPACE
OUTPUTS = {"y", "state_out", "h_out", "h_chunks", "dx", "dz", "ddt", "dBt", "dCt", "dA", "dskip", "ddt_bias", "dh0",
           "dweight", "dbias", "dstate0", "state"}


def _point(a, skip=()):
    """Gives every pointer field its own fake address; returns the names."""
    names = []

    def walk(s, prefix):
        for n, t in s._fields_:
            if isinstance(getattr(s, n), ctypes.Structure):
                walk(getattr(s, n), prefix + n + ".")
            elif t is ctypes.c_void_p and n not in skip:
                setattr(s, n, fake(len(names)))
                names.append(prefix + n)
    walk(a, "")
    return names


def _set(a, path, value):
    *head, last = path.split(".")
    for h in head:
        a = getattr(a, h)
    setattr(a, last, value)


def _get(a, path):
    for h in path.split("."):
        a = getattr(a, h)
    return a


def conv():
    a = layer.ConvArgs(B=2, T=70, C=64, x_stride=128, width=4, dtype=gdr2.BF16, act=1)
    _point(a, skip=("offsets",))
    return a


def conv_step():
    a = layer.ConvStepArgs(N=5, C=64, x_stride=64, width=4, dtype=gdr2.BF16, act=1)
    _point(a)
    return a


def conv_bwd():
    a = layer.ConvBwdArgs(B=2, T=70, C=64, x_stride=64, width=3, dtype=gdr2.F32, act=0)
    _point(a, skip=("offsets",))
    a.workspace_bytes = 1 << 30
    return a


def _scan(T=70):
    a = layer.ScanArgs(B=2, T=T, C=64, N=16, G=2, x_stride=64, dt_stride=64, b_stride=64, c_stride=64, z_stride=128,
                       dtype=gdr2.BF16, flags=1)
    return a


def scan():
    a = _scan(6400)
    a.algo = gdr2.ALGOS["segmented"]       # has a workspace
    _point(a, skip=("offsets",))
    a.workspace_bytes = 1 << 30
    return a


def scan_step():
    a = layer.ScanStepArgs(s=_scan(1))
    _point(a, skip=("offsets", "h0", "h_out", "h_chunks", "workspace"))
    return a


def scan_bwd():
    a = layer.ScanBwdArgs(f=_scan())
    _point(a, skip=("offsets",))
    a.workspace_bytes = 1 << 30
    return a


def norm():
    a = layer.NormArgs(R=7, C=64, x_stride=64, z_stride=64, dtype=gdr2.BF16, kind=0, eps=1e-5)
    _point(a)
    return a


def norm_bwd():
    a = layer.NormBwdArgs(f=layer.NormArgs(R=7, C=64, x_stride=64, z_stride=64, dtype=gdr2.F32, kind=1, eps=1e-5))
    _point(a)
    a.workspace_bytes = 1 << 30
    return a


MAKE = {"gdr2_conv_forward": conv, "gdr2_conv_step": conv_step, "gdr2_conv_backward": conv_bwd, "gdr2_scan_forward": scan,
        "gdr2_scan_step": scan_step, "gdr2_scan_backward": scan_bwd, "gdr2_norm_forward": norm,
        "gdr2_norm_backward": norm_bwd}

# fields, value, status
CASES = {
    "gdr2_conv_forward": [("B", -1, INV), ("T", -1, INV), ("C", 0, INV), ("x_stride", 63, INV), ("width", 1, UNS),
                          ("width", 5, UNS), ("dtype", 2, INV), ("act", 2, INV), ("reserved", 1, INV), ("T", 1 << 50, UNS),
                          ("B", 1 << 45, UNS), ("x_stride", 1 << 61, UNS)],
    "gdr2_conv_step": [("N", -1, INV), ("C", -3, INV), ("x_stride", 10, INV), ("width", 0, UNS), ("dtype", -1, INV),
                       ("act", -1, INV), ("reserved", 7, INV), ("N", 1 << 40, UNS)],
    "gdr2_conv_backward": [("B", -1, INV), ("width", 5, UNS), ("dtype", 9, INV), ("act", 3, INV), ("x_stride", 1, INV),
                           ("workspace_bytes", 0, WSP), ("workspace", None, WSP)],
    "gdr2_scan_forward": [("B", -2, INV), ("C", 0, INV), ("N", 0, INV), ("G", 0, INV), ("G", 3, INV), ("N", 33, UNS),
                          ("dtype", 2, INV), ("flags", 2, INV), ("algo", 3, INV), ("reserved", 1, INV), ("x_stride", 63, INV),
                          ("dt_stride", 63, INV), ("b_stride", 31, INV), ("c_stride", 0, INV), ("z_stride", 63, INV),
                          ("T", 1 << 41, UNS), ("B", 1 << 33, UNS)],
    "gdr2_scan_step": [("s.T", 2, INV), ("s.B", -1, INV), ("s.N", 40, UNS), ("s.dtype", 5, INV), ("s.h0", fake(60), INV),
                       ("s.offsets", fake(60), INV), ("s.h_out", fake(60), INV), ("s.h_chunks", fake(60), INV)],
    "gdr2_scan_backward": [("f.N", 33, UNS), ("f.G", 5, INV), ("f.algo", 9, INV), ("workspace_bytes", 16, WSP),
                           ("f.z", None, INV), ("f.c_stride", 5, INV)],
    "gdr2_norm_forward": [("R", -1, INV), ("C", 0, INV), ("x_stride", 3, INV), ("z_stride", 3, INV), ("dtype", 2, INV),
                          ("kind", 2, INV), ("eps", -1.0, INV), ("eps", float("inf"), INV), ("eps", float("nan"), INV),
                          ("reserved", 1, INV), ("R", 1 << 40, UNS)],
    "gdr2_norm_backward": [("f.C", -1, INV), ("f.kind", -1, INV), ("workspace_bytes", 0, WSP), ("f.z", None, INV)],
}
OPTIONAL = {"bias", "state0", "offsets", "state_out", "dstate", "dbias", "dstate0", "z", "f.z", "s.z", "skip", "dt_bias", "h0",
            "h_out", "h_chunks", "s.skip", "s.dt_bias", "f.skip", "f.dt_bias", "f.h0", "f.h_out", "f.y", "f.workspace",
            "workspace", "s.workspace", "dh_out", "dskip", "ddt_bias", "dh0", "weight", "f.weight", "f.bias", "dweight"}
# pointers a call does not read
IGNORED = {"gdr2_scan_backward": {"f.h0", "f.y", "f.h_out", "f.workspace"}, "gdr2_norm_backward": {"f.y"}}


def call(lib, name, a):  # noqa: F811
    return getattr(lib, name)(ctypes.byref(a), None)


@pytest.mark.parametrize("name,field,value,status", [(n, *c) for n, cs in CASES.items() for c in cs])
def test_refuses_sizes_and_modes(lib, name, field, value, status):  # noqa: F811
    a = MAKE[name]()
    _set(a, field, value)
    assert call(lib, name, a) == status, lib.gdr2_last_error()
    assert lib.gdr2_last_error()


@pytest.mark.parametrize("name", list(MAKE))
def test_refuses_null_args(lib, name):  # noqa: F811
    assert getattr(lib, name)(None, None) == INV


def _pointers(name):
    a = MAKE[name]()
    return [p for p in _point(MAKE[name](), skip=()) if _get(a, p) is not None]


def _required(name):
    conv_weight = name.startswith("gdr2_conv")
    for p in _pointers(name):
        if p in IGNORED.get(name, ()):
            continue
        last = p.split(".")[-1]
        if last in ("weight", "dweight") and conv_weight or p == "f.h_chunks" or p not in OPTIONAL:
            yield p


@pytest.mark.parametrize("name", list(MAKE))
def test_refuses_missing_pointers(lib, name):  # noqa: F811
    for p in _required(name):
        a = MAKE[name]()
        _set(a, p, None)
        assert call(lib, name, a) == INV, p
        assert p.split(".")[-1].encode() in lib.gdr2_last_error(), (p, lib.gdr2_last_error())


@pytest.mark.parametrize("name", list(MAKE))
def test_refuses_misaligned_and_overlapping(lib, name):  # noqa: F811
    ptrs = [p for p in _pointers(name) if p not in IGNORED.get(name, ())]
    rows = {"x", "dt", "Bt", "Ct", "z"}
    for i, p in enumerate(ptrs):
        a = MAKE[name]()
        _set(a, p, _get(a, p) + (1 if p.split(".")[-1] in rows else 8))
        assert call(lib, name, a) == INV and b"aligned" in lib.gdr2_last_error(), p
    pairs = 0
    for p in ptrs:
        if p.split(".")[-1] not in OUTPUTS | {"workspace"} or p == "f.h_chunks":     # the backward reads it
            continue
        for o in ptrs:
            if o == p:
                continue
            for shift in (0, 16):
                a = MAKE[name]()
                if (p, o) in (("state_out", "state0"), ("h_out", "h0"), ("dh0", "dh_out")) and shift == 0:
                    continue
                # the other buffer starts `shift` bytes into this one
                _set(a, o, _get(a, p) + shift)
                assert call(lib, name, a) == INV and b"overlaps" in lib.gdr2_last_error(), (p, o, shift, lib.gdr2_last_error())
                pairs += 1
    assert pairs


@pytest.mark.parametrize("name,alias", [("gdr2_conv_forward", ("state_out", "state0")), ("gdr2_scan_forward", ("h_out", "h0")),
                                        ("gdr2_scan_backward", ("dh0", "dh_out"))])
def test_accepts_states_in_place(lib, name, alias):  # noqa: F811
    """Passes the overlap rule (and then fails on purpose: a misaligned x
    checked first would say so, a missing one is said after the alias)."""
    a = MAKE[name]()
    _set(a, alias[0], _get(a, alias[1]))
    _set(a, "f.x" if name.endswith("backward") else "x", None)
    assert call(lib, name, a) == INV and b"x is NULL" in lib.gdr2_last_error()


def test_empty_batches_launch_nothing(lib):  # noqa: F811
    for name, field in (("gdr2_conv_forward", "B"), ("gdr2_conv_step", "N"), ("gdr2_scan_forward", "B"),
                        ("gdr2_scan_step", "s.B"), ("gdr2_norm_forward", "R")):
        a = MAKE[name]()
        _set(a, field, 0)
        assert call(lib, name, a) == gdr2.OK, (name, lib.gdr2_last_error())


def test_workspace_sizes(lib):  # noqa: F811
    a = scan()
    a.algo = gdr2.ALGOS["staged"]
    assert lib.gdr2_scan_workspace_size(ctypes.byref(a)) == 0          # one segment
    a.B, a.algo = 1, gdr2.ALGOS["segmented"]
    # 100 segments of 64 tokens: [100][C][N] states and [100][C] sums
    assert lib.gdr2_scan_workspace_size(ctypes.byref(a)) == 100 * 64 * 16 * 4 + 100 * 64 * 4
    a.N = 33
    assert lib.gdr2_scan_workspace_size(ctypes.byref(a)) == 0
    b = scan_bwd()
    # dB, dC parts of two channel blocks; sums of two sequences
    assert lib.gdr2_scan_backward_workspace_size(ctypes.byref(b)) == 2 * 140 * 2 * 16 * 4 + 2 * 64 * 18 * 4
    for make, size in ((conv_bwd, "gdr2_conv_backward_workspace_size"), (norm_bwd, "gdr2_norm_backward_workspace_size")):
        c = make()
        need = getattr(lib, size)(ctypes.byref(c))
        assert need > 0
        c.workspace_bytes = need - 1
        assert call(lib, size.replace("_workspace_size", ""), c) == WSP
        assert getattr(lib, size)(None) == 0
    assert [lib.gdr2_scan_chunk_count(*v) for v in ((2, 100, 0), (2, 64, 0), (3, 100, 1), (0, 9, 1), (2, 0, 0), (2, 0, 1))] \
        == [8, 4, 6, 0, 0, 2]


# ---- the binding's own checks (before any device is touched) ---------------

def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_conv_shapes():
    x, w = _t(2, 5, 6), _t(6, 4)
    good = dict(x=x, weight=w)
    bad = [dict(good, weight=_t(5, 4)), dict(good, x=_t(5, 6)), dict(good, bias=_t(5)), dict(good, state0=_t(2, 4, 6)),
           dict(good, out=_t(2, 5, 7)), dict(good, state_out=_t(2, 3, 5)), dict(good, x=x.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(good, x=_t(2, 7, 6)[:, :5]), dict(good, x=_t(1, 1, 6).expand(2, 5, 6)),
           dict(good, offsets=torch.zeros(3, dtype=torch.int64)), dict(good, x=_t(5, 6), offsets=torch.zeros(0, dtype=torch.int64))]
    for kw in bad:
        with pytest.raises(ValueError):
            layer.conv_forward(**kw)
    for kw in (dict(good, weight=w.double()), dict(good, x=x.half()), dict(good, state0=_t(2, 3, 6, dtype=torch.bfloat16)),
               dict(x=_t(5, 6), weight=w, offsets=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(TypeError):
            layer.conv_forward(**kw)
    with pytest.raises(ValueError, match="shape"):
        layer.conv_backward(x, w, _t(2, 5, 5))
    with pytest.raises(ValueError, match="shape"):
        layer.conv_step(_t(2, 2, 6), _t(2, 6), w)
    with pytest.raises(ValueError, match="device tensor"):
        layer.conv_forward(x, w)
    for f in (lambda: layer.conv_forward(x, w, activation="relu"), lambda: layer.conv_step(_t(2, 3, 6), _t(2, 6), w, activation="relu"),
              lambda: layer.conv_backward(x, w, x, activation="relu")):
        with pytest.raises(ValueError, match="activation"):
            f()


def test_binding_refuses_scan_shapes():
    def good():
        return dict(x=_t(2, 5, 6), dt=_t(2, 5, 6), A=_t(6, 4), Bt=_t(2, 5, 3, 4), Ct=_t(2, 5, 3, 4))
    for kw in (dict(dt=_t(2, 5, 5)), dict(A=_t(5, 4)), dict(A=_t(6)), dict(Bt=_t(2, 5, 4)), dict(Ct=_t(2, 5, 2, 4)),
               dict(z=_t(2, 4, 6)), dict(skip=_t(5)), dict(dt_bias=_t(7)), dict(h0=_t(2, 4, 6)), dict(out=_t(2, 5, 1)),
               dict(h_out=_t(1, 6, 4)), dict(chunk_states=_t(3, 6, 4)), dict(x=_t(10, 6)),
               dict(Bt=_t(2, 5, 4, 3).transpose(2, 3)[:, :, :3]), dict(offsets=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            layer.scan_forward(**{**good(), **kw})
    with pytest.raises(TypeError):
        layer.scan_forward(**{**good(), "dt": _t(2, 5, 6, dtype=torch.bfloat16)})
    with pytest.raises(ValueError, match="shape"):
        layer.scan_backward(**good(), dy=_t(2, 5, 6), h_chunks=_t(1, 6, 4))
    with pytest.raises(ValueError, match="shape"):
        layer.scan_step(_t(2, 6, 5), _t(2, 6), _t(2, 6), _t(6, 4), _t(2, 3, 4), _t(2, 3, 4))
    with pytest.raises(ValueError, match="device tensor"):
        layer.scan_forward(**good())
    with pytest.raises(ValueError, match="algo"):
        layer.scan_args(2, 5, 6, 4, 3, **good(), skip=None, z=None, dt_bias=None, softplus=True, algo="fused")


def test_binding_refuses_norm_shapes():
    x = _t(3, 4, 8)
    for kw in (dict(weight=_t(7)), dict(bias=_t(9)), dict(z=_t(3, 4, 7)), dict(out=_t(12, 8))):
        with pytest.raises(ValueError):
            layer.norm_forward(x, **kw)
    with pytest.raises(ValueError):
        layer.norm_forward(x.transpose(1, 2))
    with pytest.raises(ValueError):
        layer.norm_forward(_t(3, 0))
    with pytest.raises(TypeError):
        layer.norm_forward(x, weight=_t(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape"):
        layer.norm_backward(x, _t(3, 4, 9))
    with pytest.raises(ValueError, match="device tensor"):
        layer.norm_forward(x)


def test_row_strides():
    """What counts as equally spaced rows, and the stride found."""
    x = _t(4, 6, 32)
    assert layer._row_stride(x, "x", 2, 32) == 32
    assert layer._row_stride(x[..., 8:24], "x", 2, 16) == 32
    assert layer._row_stride(x[:, :1, :8], "x", 2, 8) == 192
    assert layer._row_stride(x[:1, ::2], "x", 2, 32) == 64
    assert layer._row_stride(x[:, ::3, :4], "x", 2, 4) == 96
    assert layer._row_stride(x[:1, :1], "x", 2, 32) == 32
    assert layer._row_stride(x[..., :24].unflatten(-1, (3, 8)), "x", 2, 24) == 32
    assert layer._row_stride(x[:0], "x", 2, 32) == 32
    for bad in (x[:, :5], x[..., ::2], x.transpose(0, 1)):
        with pytest.raises(ValueError):
            layer._row_stride(bad, "x", 2, bad.shape[-1])
    with pytest.raises(ValueError):
        layer._row_stride(x[0].unfold(1, 8, 4), "x", 2, 8)      # overlapping rows


def test_row_strides_of_expanded_rows():
    """A row repeated by expand has stride 0: taken for dense rows it would be
    read far past its end."""
    one = torch.zeros(1, 1, 8)
    for bad in (one.expand(1, 5, 8), one.expand(5, 1, 8), one.expand(4, 5, 8), torch.zeros(4, 1, 8).expand(4, 5, 8),
                torch.zeros(1, 5, 8).expand(4, 5, 8), torch.zeros(8).expand(3, 8), torch.zeros(1, 1, 1).expand(2, 3, 1)):
        with pytest.raises(ValueError):
            layer._row_stride(bad, "x", bad.dim() - 1, bad.shape[-1])
    with pytest.raises(ValueError):
        layer._row_stride(torch.zeros(4, 5, 1).expand(4, 5, 8), "x", 2, 8)      # one element for a whole row


def test_refuses_more_threads_than_one_launch_takes(lib):  # noqa: F811
    """The scan runs in workgroups of 512 threads, of 1024 for state sizes above
    16: a grid of 2^32 threads is refused here, not by the launch."""
    for N, C, B, ok in ((32, 1, 4_200_000, False), (32, 1, 4_100_000, True), (16, 1, 8_400_000, False), (16, 1, 8_300_000, True)):
        a = layer.ScanArgs(B=B, T=1, C=C, N=N, G=1, x_stride=1, dt_stride=1, b_stride=N, c_stride=N, dtype=gdr2.F32)
        status = lib.gdr2_scan_forward(ctypes.byref(a), None)       # every pointer is NULL: nothing launches
        assert status == (INV if ok else UNS), (N, B)


def test_gradient_buffers_by_name():
    dev = torch.device("cuda", 0)
    f32 = torch.float32
    for out in ({"dy": _t(2, 3)}, {"dz": _t(2, 3)}):
        with pytest.raises(ValueError, match="no gradient"):
            layer._grad_buffers(out, dev, dx=(f32, (2, 3)), dz=None)
    with pytest.raises(ValueError, match="shape"):
        layer._grad_buffers({"dx": _t(3, 2)}, dev, dx=(f32, (2, 3)))
    with pytest.raises(TypeError):
        layer._grad_buffers({"dx": _t(2, 3).bfloat16()}, dev, dx=(f32, (2, 3)))
    with pytest.raises(ValueError, match="device tensor"):
        layer._grad_buffers({"dx": _t(2, 3)}, dev, dx=(f32, (2, 3)))
