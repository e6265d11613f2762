"""GPU tests of the layer operators (convolution, scan, norm) against their
plain 64-bit implementation, at the sizes, masks and strides where they can go
wrong.  Tolerances: half a step of the stored type, plus the number of fp32
roundings a term can pass through times 2^-24 times the magnitude sum of the
terms (tests/layer_reference.py):
- convolution: at most 4 products, an activation, 32 roundings; its weight
  gradients add up rows one after the other;
- scan: every token multiplies a state by one decay, whose exponent (|d A| <=
  4 here) and exponential are off by 16 roundings, and adds two products; a
  gradient passes the recurrence twice;
- norm: the sums of a row run through C / 8 additions in sequence at most."""
import pytest
import torch

from gated_delta_rule_86_amd import gdr2, layer
from tests import layer_reference as ref
from tests.layer_reference import close

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SENT = -7.25e30
GUARD = 64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def sliced(t, extra, at):
    """The same values as a column slice of a wider matrix."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    v = wide[..., at:at + t.shape[-1]]
    v.copy_(t)
    return v


class Guarded:
    """An output inside a larger buffer of sentinels."""

    def __init__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        pad = GUARD * (4 if dtype == torch.bfloat16 else 2)
        self.buf = torch.full((n + 2 * pad,), SENT, dtype=dtype, device="cuda")
        self.pad, self.n = pad, n
        self.t = self.buf[pad:pad + n].view(shape)

    def check(self, name):
        s = torch.tensor(SENT, dtype=self.buf.dtype, device="cuda")
        assert bool((self.buf[:self.pad] == s).all()) and bool((self.buf[self.pad + self.n:] == s).all()), name


def untouched(t, offsets, T):
    """Rows of no sequence still hold the sentinel."""
    o = [int(v) for v in offsets]
    s = torch.tensor(SENT, dtype=t.dtype, device=t.device)
    return bool((t[:o[0]] == s).all()) and bool((t[o[-1]:] == s).all())


LENGTHS = [0, 1, 2, 5, 0, 33, 64, 3, 100, 0]      # packed: five rows before, seven behind


def packed():
    offs = [5]
    for n in LENGTHS:
        offs.append(offs[-1] + n)
    return torch.tensor(offs, dtype=torch.int64).cuda(), offs[-1] + 7


# ---- convolution -----------------------------------------------------------

CONV = [
    # B, T, C, K, act, packed, init, bias, slice (extra columns, first column)
    (1, 1, 1, 2, "silu", False, False, True, None),
    (2, 3, 8, 4, None, False, True, False, None),
    (3, 33, 64, 4, "silu", False, True, True, (64, 0)),
    (2, 70, 130, 3, "silu", False, False, True, (7, 3)),
    (2, 257, 72, 2, "silu", False, True, True, (8, 8)),
    (1, 2, 40, 4, "silu", False, True, True, None),
    (0, 0, 40, 4, "silu", True, True, True, None),
    (0, 0, 37, 3, None, True, False, True, (3, 2)),
    (2, 0, 16, 4, "silu", False, True, True, None),
    (9, 300, 520, 4, "silu", False, False, True, (520, 0)),
]
CONV_IDS = [f"B{c[0]}T{c[1]}C{c[2]}K{c[3]}{'p' if c[5] else ''}" for c in CONV]


def conv_case(c, dtype, seed):
    B, T, C, K, act, is_packed, init, with_bias, cut = c
    g = gen(seed)
    offsets = None
    lead = (B, T)
    if is_packed:
        offsets, T = packed()
        B, lead = len(LENGTHS), (T,)
    x = rn(g, *lead, C, dtype=DT[dtype])
    if cut:
        x = sliced(x, *cut)
    w, b = rn(g, C, K), rn(g, C) if with_bias else None
    st = rn(g, B, K - 1, C, dtype=DT[dtype]) if init else None
    return x, w, b, st, offsets, act


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", CONV, ids=CONV_IDS)
def test_conv_forward(c, dtype):
    x, w, b, st, offsets, act = conv_case(c, dtype, 11)
    B, K, C = (len(LENGTHS) if offsets is not None else c[0]), c[3], c[2]
    y, so = Guarded(x.shape, x.dtype), Guarded((B, K - 1, C), x.dtype)
    got, state = layer.conv_forward(x, w, b, st, offsets, act, out=y.t, state_out=so.t)
    torch.cuda.synchronize()
    y.check("y"), so.check("state")
    want, wst = ref.conv(x, w, b, st, offsets, act)
    bound = ref.conv(x, w, b, st, offsets, act, absolute=True)[0]
    if offsets is not None:
        assert untouched(got, offsets, x.shape[0])
        o = [int(v) for v in offsets]
        got, want, bound = (t[o[0]:o[-1]] for t in (got, want, bound))
    close(got, want, bound, 32, "y")
    assert torch.equal(state.cpu().double(), wst)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", CONV, ids=CONV_IDS)
def test_conv_backward(c, dtype):
    x, w, b, st, offsets, act = conv_case(c, dtype, 12)
    g = gen(13)
    B, K, C = (len(LENGTHS) if offsets is not None else c[0]), c[3], c[2]
    dy = rn(g, *x.shape, dtype=x.dtype)
    dst = rn(g, B, K - 1, C, dtype=x.dtype) if c[6] else None
    got = layer.conv_backward(x, w, dy, b, st, offsets, act, dstate=dst, want_dstate0=True)
    again = layer.conv_backward(x, w, dy, b, st, offsets, act, dstate=dst, want_dstate0=True)
    want = ref.conv_grad(x, w, dy, b, st, offsets, act, dst)
    bound = ref.conv_grad(x, w, dy, b, st, offsets, act, dst, absolute=True)
    rows = x.shape[0] * (x.shape[1] if offsets is None else 1)
    keep = slice(None) if offsets is None else slice(int(offsets[0]), int(offsets[-1]))
    for n in got:
        if got[n] is None:
            assert n == "dbias" and b is None
            continue
        cut = keep if n == "dx" else slice(None)
        assert torch.equal(got[n][cut], again[n][cut]), n
        close(got[n][cut], want[n][cut], bound[n][cut], 64 + (rows if n in ("dweight", "dbias") else 0), n)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,C,K,cut", [(1, 1, 2, None), (3, 64, 4, (64, 0)), (5, 37, 3, (2, 1)), (130, 264, 4, None), (0, 8, 4, None)])
def test_conv_step(N, C, K, cut, dtype):
    g = gen(14)
    x = rn(g, N, C, dtype=DT[dtype])
    if cut:
        x = sliced(x, *cut)
    w, b, st = rn(g, C, K), rn(g, C), rn(g, N, K - 1, C, dtype=DT[dtype])
    want, wst = ref.conv(x[:, None], w, b, st, None, "silu")
    bound = ref.conv(x[:, None], w, b, st, None, "silu", absolute=True)[0]
    y, s = Guarded((N, C), x.dtype), Guarded((N, K - 1, C), x.dtype)
    s.t.copy_(st)
    layer.conv_step(s.t, x, w, b, out=y.t)
    torch.cuda.synchronize()
    y.check("y"), s.check("state")
    close(y.t, want[:, 0], bound[:, 0], 32, "y")
    assert torch.equal(s.t.cpu().double(), wst)


# ---- scan ------------------------------------------------------------------

SCAN = [
    # B, T, C, N, G, packed, init, gate, extras (skip, bias), softplus, algo
    (1, 1, 1, 1, 1, False, False, False, False, True, "auto"),
    (2, 2, 3, 4, 3, False, True, True, True, True, "auto"),
    (1, 31, 65, 16, 1, False, True, True, True, True, "staged"),
    (2, 33, 64, 16, 2, False, False, True, True, True, "staged"),
    (1, 200, 40, 12, 1, False, True, False, True, True, "segmented"),
    (2, 130, 24, 16, 3, False, True, True, True, True, "segmented"),
    (1, 97, 20, 32, 1, False, True, True, True, True, "segmented"),
    (1, 64, 16, 17, 2, False, False, False, False, False, "auto"),
    (2, 96, 66, 8, 1, False, True, True, True, True, "auto"),
    (1, 1100, 6, 5, 1, False, True, True, True, True, "auto"),
    (0, 0, 20, 16, 2, True, True, True, True, True, "auto"),
    (0, 0, 20, 16, 2, True, True, True, True, True, "segmented"),
    (0, 0, 7, 3, 1, True, False, False, True, False, "staged"),
    (3, 0, 8, 16, 1, False, True, False, True, True, "auto"),
]
SCAN_IDS = [f"B{c[0]}T{c[1]}C{c[2]}N{c[3]}G{c[4]}{'p' if c[5] else ''}-{c[10]}" for c in SCAN]


def scan_case(c, dtype, seed):
    B, T, C, N, G, is_packed, init, gate, extras, softplus, algo = c
    g = gen(seed)
    offsets, lead = None, (B, T)
    if is_packed:
        offsets, T = packed()
        B, lead = len(LENGTHS), (T,)
    dt_ = DT[dtype]
    a = dict(x=sliced(rn(g, *lead, C, dtype=dt_), 5, 2), dt=rn(g, *lead, C, dtype=dt_, std=0.7),
             A=-torch.rand(C, N, generator=g).cuda() * 1.5,
             Bt=sliced(rn(g, *lead, G * N, dtype=dt_), G * N, 0).unflatten(-1, (G, N)),
             Ct=sliced(rn(g, *lead, G * N, dtype=dt_), G * N, G * N).unflatten(-1, (G, N)))
    if not softplus:
        a["dt"] = a["dt"].abs()
    kw = dict(skip=rn(g, C) if extras else None, z=sliced(rn(g, *lead, C, dtype=dt_), 3, 1) if gate else None,
              dt_bias=rn(g, C, std=0.5) - 0.5 if extras and softplus else None, offsets=offsets, softplus=softplus)
    h0 = rn(g, B, C, N) if init else None
    return a, kw, h0, B, T


def scan_steps(c, T):
    longest = max(LENGTHS) if c[5] else T
    return 64 + 32 * longest


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", SCAN, ids=SCAN_IDS)
def test_scan_forward(c, dtype):
    a, kw, h0, B, T = scan_case(c, dtype, 21)
    C, N = a["A"].shape
    y, ho = Guarded(a["x"].shape, a["x"].dtype), Guarded((B, C, N), torch.float32)
    ck = Guarded((layer.scan_chunk_count(B, T, c[5]), C, N), torch.float32)
    got, h, _ = layer.scan_forward(**a, **kw, h0=h0, out=y.t, h_out=ho.t, chunk_states=ck.t, algo=c[10])
    torch.cuda.synchronize()
    y.check("y"), ho.check("h"), ck.check("chunks")
    steps = scan_steps(c, T)
    rkw = dict(kw, offsets=None if kw["offsets"] is None else kw["offsets"].cpu())
    want, wh, marks = ref.scan(**a, **rkw, h0=h0)
    by, bh, bmarks = ref.scan(**a, **rkw, h0=h0, absolute=True)
    if c[5]:
        assert untouched(got, kw["offsets"], T)
        o = [int(v) for v in kw["offsets"]]
        got, want, by = (t[o[0]:o[-1]] for t in (got, want, by))
        first = [o[s] // 32 + s for s in range(B)]
    else:
        first = [s * -(-T // 32) for s in range(B)]
    close(got, want, by, steps, "y")
    close(h, wh, bh, steps, "h")
    for s in range(B):
        for i, (m, bm) in enumerate(zip(marks[s], bmarks[s])):
            close(ck.t[first[s] + i], m, bm, steps, f"chunk {s} {i}")
    # without the optional outputs, and in place
    if h0 is not None:
        hh = h0.clone()
        again, h2 = layer.scan_forward(**a, **kw, h0=hh, h_out=hh, out=torch.full_like(y.t, SENT), algo=c[10])
        assert torch.equal(again, y.t) and torch.equal(h2, h)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", SCAN, ids=SCAN_IDS)
def test_scan_backward(c, dtype):
    a, kw, h0, B, T = scan_case(c, dtype, 22)
    C, N = a["A"].shape
    g = gen(23)
    dy = rn(g, *a["x"].shape, dtype=a["x"].dtype)
    dh = rn(g, B, C, N) if c[6] else None
    _, _, ck = layer.scan_forward(**a, **kw, h0=h0, chunk_states=True, algo=c[10])
    got = layer.scan_backward(**a, **kw, dy=dy, h_chunks=ck, dh_out=dh, algo=c[10])
    again = layer.scan_backward(**a, **kw, dy=dy, h_chunks=ck, dh_out=dh, algo=c[10])
    rkw = dict(kw, offsets=None if kw["offsets"] is None else kw["offsets"].cpu())
    want = ref.scan_grad(**a, **rkw, dy=dy, h0=h0, dh_out=dh)
    bound = ref.scan_grad(**a, **rkw, dy=dy, h0=h0, dh_out=dh, absolute=True)
    rows = slice(None) if not c[5] else slice(int(kw["offsets"][0]), int(kw["offsets"][-1]))
    steps = 2 * scan_steps(c, T) + a["x"].shape[0] * (1 if c[5] else T)
    for n in got:
        if got[n] is None:
            assert n == "dz" and kw["z"] is None or n == "dskip" and kw["skip"] is None or n == "ddt_bias" and kw["dt_bias"] is None
            continue
        cut = rows if n in ("dx", "ddt", "dBt", "dCt", "dz") else slice(None)
        assert torch.equal(got[n][cut], again[n][cut]), n
        close(got[n][cut], want[n][cut], bound[n][cut], steps, n)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,C,N,G,gate", [(1, 1, 1, 1, False), (2, 40, 16, 2, True), (5, 37, 4, 1, True), (3, 66, 7, 3, False),
                                          (2, 30, 32, 1, True), (3, 10, 19, 2, True), (0, 8, 16, 1, False)])
def test_scan_step(B, C, N, G, gate, dtype):
    c = (B, 1, C, N, G, False, True, gate, True, True, "auto")
    a, kw, h0, _, _ = scan_case(c, dtype, 24)
    want, wh, _ = ref.scan(**a, **kw, h0=h0)
    by, bh, _ = ref.scan(**a, **kw, h0=h0, absolute=True)
    tok = {n: (t if n == "A" else t[:, 0]) for n, t in a.items()}
    y, s = Guarded((B, C), a["x"].dtype), Guarded((B, C, N), torch.float32)
    s.t.copy_(h0)
    layer.scan_step(s.t, **tok, skip=kw["skip"], z=kw["z"][:, 0] if gate else None, dt_bias=kw["dt_bias"], out=y.t)
    torch.cuda.synchronize()
    y.check("y"), s.check("state")
    close(y.t, want[:, 0], by[:, 0], 128, "y")
    close(s.t, wh, bh, 128, "state")


def test_scan_small_and_large_steps():
    """softplus keeps its relative accuracy over its whole range: a state of
    one token is d x B with nothing else in it."""
    raw = torch.linspace(-60, 60, 481).cuda()
    x = torch.ones(1, 1, 481).cuda()
    one = torch.ones(1, 1, 1, 1).cuda()
    _, h = layer.scan_forward(x, raw.view(1, 1, -1), torch.zeros(481, 1).cuda(), one, one)
    want = torch.nn.functional.softplus(raw.cpu().double(), threshold=100)
    close(h.view(-1), want, want.abs(), 16, "softplus")


# ---- norm ------------------------------------------------------------------

WIDTHS = [1, 7, 8, 64, 100, 128, 130, 256, 513, 1000, 1003, 1024, 2048, 2056, 4096, 5000, 8192, 8200, 16384, 16392, 20001]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", WIDTHS)
def test_norm(C, dtype, kind):
    g = gen(31 + C)
    R = 3 if C > 2000 else 37
    gate, affine, with_bias = C % 3 != 0, C != 64, kind == "layer"
    x = rn(g, R, C, dtype=DT[dtype]) * 1.5 + 0.5
    x = sliced(x, C, 0) if C % 2 == 0 else x
    z = sliced(rn(g, R, C, dtype=DT[dtype]), C, C) if gate else None
    w, b = (1 + 0.2 * rn(g, C) if affine else None), (rn(g, C) if affine and with_bias else None)
    dy = rn(g, R, C, dtype=DT[dtype])
    y = Guarded((R, C), DT[dtype])
    layer.norm_forward(x, w, b, z, kind=kind, out=y.t)
    got = layer.norm_backward(x, dy, w, b, z, kind=kind)
    again = layer.norm_backward(x, dy, w, b, z, kind=kind)
    torch.cuda.synchronize()
    y.check("y")
    steps = 64 + C / 8
    want, bound = ref.norm(x, w, b, z, kind=kind)
    close(y.t, want, bound, steps, "y")
    wg, bg = ref.norm_grad(x, dy, w, b, z, kind=kind)
    for n in got:
        if got[n] is None:
            assert n == "dz" and z is None or n == "dweight" and w is None or n == "dbias" and b is None
            continue
        assert torch.equal(got[n], again[n]), n
        close(got[n], wg[n], bg[n], 2 * steps + R, n)


def test_norm_leading_dims_and_many_rows():
    g = gen(32)
    x = rn(g, 3, 700, 2, 128, dtype=torch.bfloat16)
    w = rn(g, 128)
    dy, z = rn(g, *x.shape, dtype=x.dtype), rn(g, *x.shape, dtype=x.dtype)
    y = layer.norm_forward(x, w, None, z, kind="rms")
    want, bound = ref.norm(x, w, None, z, kind="rms")
    close(y, want, bound, 128, "y")
    got = layer.norm_backward(x, dy, w, None, z, kind="rms")
    wg, bg = ref.norm_grad(x, dy, w, None, z, kind="rms")
    for n in ("dx", "dz", "dweight"):
        close(got[n], wg[n], bg[n], 256 + 4200, n)


def test_norm_of_no_rows():
    x = torch.zeros(0, 64).cuda()
    w = torch.ones(64).cuda()
    assert layer.norm_forward(x, w).shape == (0, 64)
    g = layer.norm_backward(x, x, w, w)
    torch.cuda.synchronize()
    assert bool((g["dweight"] == 0).all()) and bool((g["dbias"] == 0).all())


# ---- variants that only larger or aligned calls reach ----------------------

WIDE = [
    # B, T, C, N, G: rows aligned to whole vectors, contiguous or as aligned slices
    (2, 77, 64, 16, 1), (1, 130, 128, 16, 2), (2, 45, 72, 8, 1), (1, 70, 24, 32, 1), (3, 33, 200, 13, 1),
]


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("B,T,C,N,G", WIDE)
def test_scan_aligned_rows(B, T, C, N, G, dtype, gate):
    g = gen(71)
    dt_ = DT[dtype]
    a = dict(x=sliced(rn(g, B, T, C, dtype=dt_), C, 0), dt=rn(g, B, T, C, dtype=dt_, std=0.7),
             A=-torch.rand(C, N, generator=g).cuda() * 1.5, Bt=rn(g, B, T, G, N, dtype=dt_), Ct=rn(g, B, T, G, N, dtype=dt_))
    kw = dict(skip=rn(g, C), z=sliced(rn(g, B, T, C, dtype=dt_), C, C) if gate else None, dt_bias=rn(g, C, std=0.5))
    h0, dy, dh = rn(g, B, C, N), rn(g, B, T, C, dtype=dt_), rn(g, B, C, N)
    y, h, ck = layer.scan_forward(**a, **kw, h0=h0, chunk_states=True)
    got = layer.scan_backward(**a, **kw, dy=dy, h_chunks=ck, dh_out=dh)
    steps = 64 + 32 * T
    want, wh, _ = ref.scan(**a, **kw, h0=h0)
    by, bh, _ = ref.scan(**a, **kw, h0=h0, absolute=True)
    close(y, want, by, steps, "y")
    close(h, wh, bh, steps, "h")
    wg = ref.scan_grad(**a, **kw, dy=dy, h0=h0, dh_out=dh)
    bg = ref.scan_grad(**a, **kw, dy=dy, h0=h0, dh_out=dh, absolute=True)
    for n in got:
        if got[n] is not None:
            close(got[n], wg[n], bg[n], 2 * steps + B * T, n)


def test_scan_step_of_many_sequences():
    """Enough sequences that a thread takes two, an odd number of them."""
    B, C, N = 33, 8200, 16
    g = gen(72)
    tok = dict(x=rn(g, B, C), dt=rn(g, B, C), A=-torch.rand(C, N, generator=g).cuda(), Bt=rn(g, B, 1, N), Ct=rn(g, B, 1, N))
    s = rn(g, B, C, N)
    s0 = s.clone()
    y = layer.scan_step(s, **tok)
    one = s0.clone()
    for b in range(B):       # one at a time: the same operations on the same values
        r = {n: (t if n == "A" else t[b:b + 1]) for n, t in tok.items()}
        assert torch.equal(layer.scan_step(one[b:b + 1], **r)[0], y[b])
    assert torch.equal(one, s)
    b = B - 1
    want, wh, _ = ref.scan(**{n: (t if n == "A" else t[b:, None]) for n, t in tok.items()}, h0=s0[b:])
    by, bh, _ = ref.scan(**{n: (t if n == "A" else t[b:, None]) for n, t in tok.items()}, h0=s0[b:], absolute=True)
    close(y[b:], want[:, 0], by[:, 0], 128, "y")
    close(s[b:], wh, bh, 128, "state")


@pytest.mark.parametrize("R,C,dtype,gate", [(70001, 16, "f32", False), (2501, 2048, "bf16", False), (2100, 1500, "f32", True),
                                            (1100, 2048, "bf16", True)])
def test_norm_walks_its_rows(R, C, dtype, gate):
    """More rows than groups of lanes: each walks several."""
    g = gen(73)
    x, dy = rn(g, R, C, dtype=DT[dtype]), rn(g, R, C, dtype=DT[dtype])
    z = rn(g, R, C, dtype=DT[dtype]) if gate else None
    w, b = 1 + 0.2 * rn(g, C), rn(g, C)
    want, bound = ref.norm(x, w, b, z)
    close(layer.norm_forward(x, w, b, z), want, bound, 64 + C / 8, "y")
    got = layer.norm_backward(x, dy, w, b, z)
    wg, bg = ref.norm_grad(x, dy, w, b, z)
    for n in got:
        if got[n] is not None:
            close(got[n], wg[n], bg[n], 128 + C / 4 + R, n)


def test_conv_of_a_training_batch_equals_its_channel_slices():
    """The longest pieces against the shorter ones that a slice of the channels
    takes: rows bit for bit, the taps' sums to their rounding."""
    B, T, C = 4, 4100, 2048
    g = gen(74)
    x, dy = rn(g, B, T, C, dtype=torch.bfloat16), rn(g, B, T, C, dtype=torch.bfloat16)
    w, b = rn(g, C, 4) * 0.5, rn(g, C)
    y, st = layer.conv_forward(x, w, b)
    full = layer.conv_backward(x, w, dy, b)
    for c in (slice(0, 64), slice(1000, 1072), slice(2040, 2048)):
        ys, ss = layer.conv_forward(x[..., c], w[c].contiguous(), b[c].contiguous())
        assert torch.equal(ys, y[..., c]) and torch.equal(ss, st[..., c])
        part = layer.conv_backward(x[..., c], w[c].contiguous(), dy[..., c].contiguous(), b[c].contiguous())
        assert torch.equal(part["dx"], full["dx"][..., c])
        bound = ref.conv_grad(x[..., c], w[c], dy[..., c], b[c], None, None, "silu", absolute=True)
        for n in ("dweight", "dbias"):
            close(full[n][c], ref.d64(part[n]), bound[n], 2 * (64 + B * T), n)


def test_rows_past_32_bits():
    """More than 2^31 elements: the last rows come out as they do from a call
    of their own that starts from the state before them."""
    T, C, N, tail = 1_060_000, 2048, 4, 97
    g = torch.Generator(device="cuda").manual_seed(75)
    x = torch.randn(1, T, C, generator=g, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 1 << 31
    w = torch.rand(C, 4, generator=g, device="cuda") - 0.5
    end = x[:, T - tail:].contiguous()
    y, _ = layer.conv_forward(x, w)
    again, _ = layer.conv_forward(end, w, state0=x[:, T - tail - 3:T - tail].contiguous())
    assert torch.equal(y[:, T - tail:], again)
    n = layer.norm_forward(x, kind="rms", out=y)
    assert torch.equal(n[:, T - tail:], layer.norm_forward(end, kind="rms"))
    A = -torch.rand(C, N, generator=g, device="cuda") - 0.5
    Bt = torch.randn(1, T, 1, N, generator=g, device="cuda", dtype=torch.bfloat16)
    y, h = layer.scan_forward(x, x, A, Bt, Bt, out=y)
    # the state before the tail has forgotten everything older than 3000 tokens (exp(-0.5 * 0.31 * 3000) at most)
    near = slice(T - tail - 3000, T - tail)
    _, h0 = layer.scan_forward(x[:, near], x[:, near], A, Bt[:, near], Bt[:, near])
    again, h1 = layer.scan_forward(end, end, A, Bt[:, T - tail:], Bt[:, T - tail:], h0=h0)
    assert float((h - h1).abs().max()) <= 1e-4 * float(h.abs().max())
    assert float((y[:, T - tail:].float() - again.float()).abs().max()) <= 2.0 ** -7 * float(again.float().abs().max())


def test_empty_packed_batches():
    """Only empty sequences, with and without rows around them; no sequence."""
    for T, offs in ((0, [0, 0, 0]), (9, [4, 4, 4]), (9, [3]), (0, [0])):
        offsets = torch.tensor(offs, dtype=torch.int64).cuda()
        B = len(offs) - 1
        g = gen(76)
        x, w = rn(g, T, 8), rn(g, 8, 4)
        st, h0 = rn(g, B, 3, 8), rn(g, B, 8, 4)
        y, s = layer.conv_forward(x, w, state0=st, offsets=offsets, out=torch.full_like(x, SENT))
        assert torch.equal(s, st) and bool((y == SENT).all())
        gc = layer.conv_backward(x, w, x, w[:, 0].contiguous(), state0=st, offsets=offsets, dstate=st)
        assert bool((gc["dweight"] == 0).all()) and bool((gc["dbias"] == 0).all()) and torch.equal(gc["dstate0"], st)
        A, bc = -torch.ones(8, 4).cuda(), rn(g, T, 1, 4)
        y, h, ck = layer.scan_forward(x, x, A, bc, bc, h0=h0, offsets=offsets, chunk_states=True, out=torch.full_like(x, SENT))
        assert torch.equal(h, h0) and bool((y == SENT).all())
        gs = layer.scan_backward(x, x, A, bc, bc, x, ck, offsets=offsets, dh_out=h0)
        assert bool((gs["dA"] == 0).all()) and torch.equal(gs["dh0"], h0)


# ---- what no sequence owns, and bad values ---------------------------------

def test_values_outside_the_sequences_do_not_matter():
    """NaN and infinities in rows of no sequence, and in one sequence, stay there."""
    offsets, T = packed()
    o = [int(v) for v in offsets]
    c = SCAN[10]
    a, kw, h0, B, _ = scan_case(c, "bf16", 41)
    g = gen(42)
    dy = rn(g, *a["x"].shape, dtype=a["x"].dtype)

    def all_of(a, kw, dy):
        y, h, ck = layer.scan_forward(**a, **kw, h0=h0, chunk_states=True)
        r = layer.scan_backward(**a, **kw, dy=dy, h_chunks=ck)
        w = torch.linspace(-1, 1, 20 * 4).view(20, 4).cuda()
        cy, cs = layer.conv_forward(a["x"], w, None, None, offsets)
        cg = layer.conv_backward(a["x"], w, dy, None, None, offsets)
        return {"y": y, "h": h, **r, "cy": cy, "cs": cs, "cdx": cg["dx"], "cdw": cg["dweight"]}

    clean = all_of(a, kw, dy)
    for rows in (slice(0, o[0]), slice(o[-1], T)):
        for t in (a["x"], a["dt"], a["Bt"], a["Ct"], kw["z"], dy):
            t[rows] = float("nan")
        a["x"][rows] = float("inf")
    dirty = all_of(a, kw, dy)
    rowed = {"y", "dx", "ddt", "dBt", "dCt", "dz", "cy", "cdx"}
    for n in clean:
        if clean[n] is None:
            continue
        cut = slice(o[0], o[-1]) if n in rowed else slice(None)
        assert torch.equal(clean[n][cut], dirty[n][cut]), n
    # one sequence turns to NaN: the others' rows and states do not
    s = 5
    a["x"][o[s]] = float("nan")
    dirty = all_of(a, kw, dy)
    for n in clean:
        if n in rowed:
            keep = torch.cat([clean[n][o[0]:o[s]], clean[n][o[s + 1]:o[-1]]])
            assert torch.equal(keep, torch.cat([dirty[n][o[0]:o[s]], dirty[n][o[s + 1]:o[-1]]])), n
        elif n in ("h", "cs"):
            assert torch.equal(torch.cat([clean[n][:s], clean[n][s + 1:]]), torch.cat([dirty[n][:s], dirty[n][s + 1:]])), n
    assert bool(dirty["y"][o[s]].isnan().any())


def test_scan_small_and_large_steps_of_bf16_rows():
    """bf16 rows form softplus with its exponent x log2(e) as rounded: one
    rounding of the product and one of the constant, each 2^-24 |x| of the
    result at most, beside the 16 of the rest."""
    raw = torch.linspace(-60, 60, 481).bfloat16().cuda()
    x, one = torch.ones(1, 1, 481).bfloat16().cuda(), torch.ones(1, 1, 1, 1).bfloat16().cuda()
    _, h = layer.scan_forward(x, raw.view(1, 1, -1), torch.zeros(481, 1).cuda(), one, one)
    want = torch.nn.functional.softplus(raw.cpu().double(), threshold=100)
    close(h.view(-1), want, want.abs(), 16 + 2 * 60, "softplus")


@pytest.mark.parametrize("algo", ["staged", "segmented"])
def test_infinite_decay(algo):
    """A = -inf (and values whose multiple by log2(e) overflows) forgets the
    state at every step, as any large finite decay does: also at the tokens
    that fill up the last chunk, and in the gradients."""
    B, T, C, N = 2, 70, 5, 6
    g = gen(44)
    x, dt, bc = rn(g, B, T, C), rn(g, B, T, C).abs() + 0.25, rn(g, B, T, 1, N)
    h0, dy = rn(g, B, C, N), rn(g, B, T, C)
    A = -torch.rand(C, N, generator=g).cuda()
    A[:, 1], A[:, 4] = -float("inf"), -3e38
    big = A.clone()
    big[:, 1] = big[:, 4] = -1e6                     # exp(-0.25e6) is 0 in every format
    res = []
    for a in (A, big):
        y, h, ck = layer.scan_forward(x, dt, a, bc, bc, h0=h0, softplus=False, chunk_states=True, algo=algo)
        res.append({"y": y, "h": h, **layer.scan_backward(x, dt, a, bc, bc, dy, ck, softplus=False, algo=algo)})
    for n, want in res[1].items():
        if want is not None:
            assert bool(want.isfinite().all()) and torch.equal(res[0][n], want), n


def test_gradients_into_given_buffers():
    """Rows of no sequence keep what the given buffers hold there; the rest is
    what a call without buffers returns."""
    offsets, T = packed()
    lo, hi = int(offsets[0]), int(offsets[-1])
    a, kw, h0, B, _ = scan_case(SCAN[10], "bf16", 45)
    dy = rn(gen(46), *a["x"].shape, dtype=a["x"].dtype)
    _, _, ck = layer.scan_forward(**a, **kw, h0=h0, chunk_states=1)
    w = torch.linspace(-1, 1, 20 * 4).view(20, 4).cuda()
    calls = {("dx", "ddt", "dBt", "dCt", "dz"): lambda o: layer.scan_backward(**a, **kw, dy=dy, h_chunks=ck, out=o),
             ("dx",): lambda o: layer.conv_backward(a["x"], w, dy, offsets=offsets, out=o)}
    for names, call in calls.items():
        want = call(None)
        given = {n: torch.full_like(want[n], SENT) for n in names}
        got = call(given)
        for n in names:
            assert got[n] is given[n] and untouched(got[n], offsets, T) and torch.equal(got[n][lo:hi], want[n][lo:hi]), n
    wn = torch.ones(20).cuda()
    want, given = layer.norm_backward(dy, dy, wn), {"dx": torch.empty_like(dy), "dweight": torch.empty_like(wn)}
    got = layer.norm_backward(dy, dy, wn, out=given)
    assert all(got[n] is given[n] and torch.equal(got[n], want[n]) for n in given)


def test_bad_offsets_stay_inside():
    """Offsets out of range or descending are clamped on the device: the call
    returns and writes only its outputs' rows."""
    g = gen(43)
    x, w = rn(g, 50, 8), rn(g, 8, 4)
    for offs in ([-5, 20, 90], [40, 10, 50], [0, 1 << 60, -(1 << 60)], [50, 50, 50], [60, 60, 60]):
        o = torch.tensor(offs, dtype=torch.int64).cuda()
        y = Guarded(x.shape, x.dtype)
        layer.conv_forward(x, w, offsets=o, out=y.t)
        h = Guarded((2, 8, 4), torch.float32)
        yy = Guarded(x.shape, x.dtype)
        bc = rn(g, 50, 1, 4)
        ck = Guarded((layer.scan_chunk_count(2, 50, True), 8, 4), torch.float32)
        layer.scan_forward(x, x, -torch.ones(8, 4).cuda(), bc, bc, offsets=o, out=yy.t, h_out=h.t, chunk_states=ck.t,
                           algo="segmented")
        layer.scan_backward(x, x, -torch.ones(8, 4).cuda(), bc, bc, x, torch.zeros_like(ck.t), offsets=o, algo="segmented")
        layer.conv_backward(x, w, x, offsets=o)
        torch.cuda.synchronize()
        for b, n in ((y, "y"), (yy, "scan"), (h, "h"), (ck, "chunks")):
            b.check(n)


# ---- a run of them together ------------------------------------------------

def mixer(p, u, states=None, offsets=None):
    """One mixing layer as a model runs it: layer norm, input projection,
    convolution, scan with its gate, rms norm."""
    C, N = p["A"].shape
    n = layer.norm_forward(u, p["nw"], p["nb"])
    proj = (n.float() @ p["win"]).to(u.dtype)
    x, z = proj[..., :C], proj[..., C:]
    st0, h0 = states if states else (None, None)
    step = u.dim() == 2 and offsets is None
    if step:
        xc = layer.conv_step(st0, x, p["cw"], p["cb"])
    else:
        xc, st0 = layer.conv_forward(x, p["cw"], p["cb"], st0, offsets)
    dbl = (xc.float() @ p["wx"]).to(u.dtype)
    Bt, Ct, dt = dbl[..., :N].unflatten(-1, (1, N)), dbl[..., N:2 * N].unflatten(-1, (1, N)), dbl[..., 2 * N:]
    kw = dict(skip=p["skip"], z=z, dt_bias=p["bias"])
    if step:
        y = layer.scan_step(h0, xc, dt, p["A"], Bt, Ct, **kw)
    else:
        y, h0 = layer.scan_forward(xc, dt, p["A"], Bt, Ct, h0=h0, offsets=offsets, **kw)
    return layer.norm_forward(y, p["ow"], kind="rms"), (st0, h0)


def mixer_params(C, N):
    g = gen(51)
    return dict(nw=1 + 0.1 * rn(g, C), nb=0.1 * rn(g, C), win=rn(g, C, 2 * C) / C ** 0.5, cw=rn(g, C, 4) * 0.5, cb=0.1 * rn(g, C),
                wx=rn(g, C, 2 * N + C) / C ** 0.5, A=-torch.rand(C, N, generator=g).cuda() - 0.2, skip=rn(g, C),
                bias=rn(g, C) - 2, ow=1 + 0.1 * rn(g, C))


def test_layer_prompt_then_tokens():
    """A prompt in two segments, then tokens one by one, equals one prompt;
    packed and dense batches agree."""
    C, N, B, T = 64, 16, 3, 150
    p = mixer_params(C, N)
    u = rn(gen(52), B, T, C)
    whole, (st, h) = mixer(p, u)
    y1, s = mixer(p, u[:, :67].contiguous())
    y2, s = mixer(p, u[:, 67:140].contiguous(), s)
    tokens = []
    for t in range(140, T):
        y, s = mixer(p, u[:, t].contiguous(), s)
        tokens.append(y[:, None])
    # the same fp32 operations but for the segments' boundaries: states agree to their rounding
    for a, b in ((torch.cat([y1, y2, *tokens], 1), whole), (s[0], st), (s[1], h)):
        assert float((a - b).abs().max()) <= 2e-4 * float(b.abs().max())
    offs = torch.arange(0, B * T + 1, T).cuda()
    flat, (pst, ph) = mixer(p, u.view(B * T, C), offsets=offs)
    for a, b in ((flat.view(B, T, C), whole), (pst, st), (ph, h)):
        assert float((a - b).abs().max()) <= 2e-4 * float(b.abs().max())


def test_with_the_gated_delta_rule():
    """Convolved q, k, v through the chunked forward and the gated head norm,
    against the reference operators around the library's own forward."""
    B, T, H, D = 2, 80, 2, 64
    g = gen(53)
    x = rn(g, B, T, 3 * H * D, dtype=torch.bfloat16)
    w = rn(g, 3 * H * D, 4) * 0.5
    qkv, _ = layer.conv_forward(x, w)
    close(qkv, *(ref.conv(x, w, None, None, None, "silu", absolute=ab)[0] for ab in (False, True)), 32, "qkv")
    q, k, v = (qkv[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).contiguous() for i in range(3))
    b, wg = (torch.rand(B, T, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    gd = -torch.rand(B, T, H, D, generator=g).cuda()
    o, _ = gdr2.forward(q, k, v, b, wg, gd, prologue=gdr2.PROLOGUE_NORM_QK)
    z, ow = rn(g, B, T, H, D, dtype=torch.bfloat16), 1 + 0.1 * rn(g, D)
    y = layer.norm_forward(o, ow, None, z, kind="rms")
    close(y, *ref.norm(o, ow, None, z, kind="rms"), 128, "y")


def test_training_step_of_the_layer():
    """Gradients through norm, convolution and scan, chained by hand, against
    the reference's chain on the same intermediate rows."""
    C, N, B, T = 40, 16, 2, 75
    g = gen(54)
    u, cw, cb = rn(g, B, T, C), rn(g, C, 4) * 0.5, rn(g, C)
    A, skip, bias = -torch.rand(C, N, generator=g).cuda(), rn(g, C), rn(g, C) - 1
    dt, z, Bt, Ct = rn(g, B, T, C), rn(g, B, T, C), rn(g, B, T, 1, N), rn(g, B, T, 1, N)
    nw, nb, dy = 1 + 0.1 * rn(g, C), rn(g, C), rn(g, B, T, C)
    n = layer.norm_forward(u, nw, nb)
    xc, _ = layer.conv_forward(n, cw, cb)
    _, _, ck = layer.scan_forward(xc, dt, A, Bt, Ct, skip, z, bias, chunk_states=True)
    gs = layer.scan_backward(xc, dt, A, Bt, Ct, dy, ck, skip, z, bias)
    gc = layer.conv_backward(n, cw, gs["dx"], cb)
    gn = layer.norm_backward(u, gc["dx"], nw, nb)
    un = ref.d64(u).requires_grad_()
    wn = ref.d64(nw).requires_grad_()
    m = un.mean(-1, keepdim=True)
    nn = (un - m) * ((un - m).square().mean(-1, keepdim=True) + 1e-5).rsqrt() * wn + ref.d64(nb)
    pad = torch.cat([torch.zeros(B, 3, C, dtype=torch.float64), nn], 1)
    xx = ref.silu(sum(pad[:, k:k + T] * ref.d64(cw)[:, k] for k in range(4)) + ref.d64(cb))
    h, outs = torch.zeros(B, C, N, dtype=torch.float64), []
    d = torch.nn.functional.softplus(ref.d64(dt) + ref.d64(bias))
    for t in range(T):
        h = torch.exp(d[:, t, :, None] * ref.d64(A)) * h + (d[:, t] * xx[:, t])[..., None] * ref.d64(Bt)[:, t]
        outs.append(((h * ref.d64(Ct)[:, t]).sum(-1) + ref.d64(skip) * xx[:, t]) * ref.silu(ref.d64(z)[:, t]))
    (torch.stack(outs, 1) * ref.d64(dy)).sum().backward()
    # three chained fp32 passes: the first norm's rounding is amplified by the later ones' slopes
    for got, want in ((gn["dx"], un.grad), (gn["dweight"], wn.grad)):
        assert float((ref.d64(got) - want).abs().max()) <= 1e-4 * float(want.abs().max())


# ---- streams and graphs ----------------------------------------------------

def test_other_stream():
    c = SCAN[5]
    a, kw, h0, _, _ = scan_case(c, "f32", 61)
    want, _ = layer.scan_forward(**a, **kw, h0=h0, algo="segmented")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, _ = layer.scan_forward(**a, **kw, h0=h0, algo="segmented")
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("algo", ["staged", "segmented"])
def test_two_calls_at_once(algo):
    """Calls on two streams, each with memory of its own, do not meet; state
    sizes of both workgroup sizes."""
    cases = [scan_case((3, 300, 130, N, 1, False, True, True, True, True, algo), "bf16", 64 + N) for N in (16, 32)]
    dys = [rn(gen(66), *a["x"].shape, dtype=a["x"].dtype) for a, *_ in cases]

    def work(i):
        a, kw, h0, _, _ = cases[i]
        y, h, ck = layer.scan_forward(**a, **kw, h0=h0, chunk_states=True, algo=algo)
        return [y, h, *(v for v in layer.scan_backward(**a, **kw, dy=dys[i], h_chunks=ck, algo=algo).values())]

    want = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for res in got[i]:
            assert all(torch.equal(g, w) for g, w in zip(res, want[i]))


def test_captured_and_replayed():
    """Forward and backward of all three in one graph, replayed on new inputs
    with eager work between the replays."""
    c = SCAN[5]
    a, kw, h0, _, _ = scan_case(c, "bf16", 62)
    C = a["A"].shape[0]
    g = gen(63)
    w, cw = 1 + 0.1 * rn(g, C), rn(g, C, 4)
    dy = rn(g, *a["x"].shape, dtype=a["x"].dtype)

    def work():
        n = layer.norm_forward(a["x"], w)
        x, st = layer.conv_forward(n, cw)
        y, h, ck = layer.scan_forward(**{**a, "x": x}, **kw, h0=h0, chunk_states=True, algo="segmented")
        gs = layer.scan_backward(**{**a, "x": x}, **kw, dy=dy, h_chunks=ck, algo="segmented")
        gc = layer.conv_backward(n, cw, gs["dx"])
        gn = layer.norm_backward(a["x"], gc["dx"], w)
        return [y, h, st, gs["dA"], gs["dBt"], gs["dz"], gs["dskip"], gc["dweight"], gn["dx"], gn["dweight"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        a["x"].copy_(rn(g, *a["x"].shape, dtype=a["x"].dtype))
        dy.copy_(rn(g, *dy.shape, dtype=dy.dtype))
        graph.replay()
        torch.cuda.synchronize()
        for n, (got, want) in enumerate(zip(out, work())):
            assert torch.equal(got, want), (i, n)
