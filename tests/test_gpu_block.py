"""GPU tests of the block operators (rows in 8 bits, norm with the residual's
addition, gated linear recurrence) against their plain 64-bit implementation,
at the sizes, masks and strides where they can go wrong.  Tolerances: half a
step of the stored type, plus the number of fp32 roundings a term can pass
through times 2^-24 times the magnitude sum of the terms:
- rows in 8 bits, from rows or from the 64-bit norm: none, codes and scales are equal;
- norm: 64-bit, so half a step (fp32: one) of the stored type; its gradients
  are fp32, the sums of a row run through C / 8 additions at most in sequence,
  those of a column through the rows;
- recurrence: s(r) is off by (2 |r| + 5) roundings (the exponent's product,
  exponential, sum, reciprocal), |r| <= 5 here; a, whose exponent is at most 1
  in magnitude, by that and 4; q by half of it and 8 (the difference loses two
  bits); a token multiplies the state once, in a product of decays or by
  itself, and adds one input: 64 per token of the bounds below cover it.  The
  gradients pass one more such factor, q's derivative (1/q off as q): 192."""
import math

import pytest
import torch

from gated_delta_rule_86_amd import block
from tests import block_reference as ref
from tests.layer_reference import close, half_step
from tests.test_gpu_layer import DT, SENT, Guarded, gen, rn, sliced

pytestmark = pytest.mark.gpu


class Guarded8:
    """Rows in 8 bits inside larger buffers of sentinels."""

    def __init__(self, shape):
        nb = -(-shape[-1] // 32)
        self.parts = []
        for width in (shape[-1], nb):
            n = width
            for s in shape[:-1]:
                n *= s
            self.parts.append((torch.full((n + 128,), 0x5A, dtype=torch.uint8, device="cuda"), n))
        (c, nc), (s, ns) = self.parts
        self.t = block.Rows8(c[64:64 + nc].view(torch.float8_e4m3fn).view(shape),
                             s[64:64 + ns].view(torch.float8_e8m0fnu).view(*shape[:-1], nb))

    def check(self, name):
        for b, n in self.parts:
            assert bool((b[:64] == 0x5A).all()) and bool((b[64 + n:] == 0x5A).all()), name


def same_rows8(got, codes, exps, name=""):
    """Codes equal as values (every NaN alike), scales as exponents."""
    assert torch.equal(got.scales.cpu().view(torch.uint8).long() - 127, exps), name
    c = got.codes.cpu().double()
    assert torch.equal(torch.isnan(c), torch.isnan(codes)), name
    keep = ~torch.isnan(codes)
    assert torch.equal(c[keep], codes[keep]), name


# ---- rows in 8 bits --------------------------------------------------------

ROWS8 = [(1, 1, None), (3, 31, None), (2, 32, None), (5, 33, (3, 2)), (4, 40, (24, 8)), (7, 64, (64, 64)), (3, 100, None), (2, 1003, (5, 1)),
         (9, 1024, None), (130, 256, None), (0, 64, None), (2, 72, (8, 0))]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("R,C,cut", ROWS8)
def test_rows8(R, C, cut, dtype):
    g = gen(31)
    x = (torch.randn(R, C, generator=g) * torch.exp2(torch.randn(R, 1, generator=g) * 4)).to(DT[dtype])
    if C > 40 and R > 1:
        x[0, 32:40], x[1, :32] = 0.0, 0.0
        x[0, 40] = 448 * 2.0 ** -7                       # on the border of a scale
        x[1, 33], x[1, 34] = 2.0 ** -60, 2.0 ** 60       # the smaller one goes to 0
    want = ref.pack(x)
    xd = x.cuda() if cut is None else sliced(x.cuda(), *cut)
    out = Guarded8((R, C))
    got = block.pack_rows(xd, out=out.t)
    torch.cuda.synchronize()
    out.check("pack")
    same_rows8(got, want[0], want[1])
    for t in (torch.float32, torch.bfloat16):
        back = Guarded((R, C), t)
        block.unpack_rows(got, t, out=back.t)
        torch.cuda.synchronize()
        back.check("unpack")
        assert torch.equal(back.t.cpu().double(), want[2].to(t).double())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", [64, 67])
def test_rows8_ties_and_ends(C, dtype):
    """Every middle between two codes, subnormal codes, the types' ends."""
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mids = (grid[:-1] + grid[1:]) / 2
    v = torch.cat([grid, mids, -grid, -mids])
    v = torch.cat([v, torch.zeros(-v.numel() % C)]).view(-1, C).clone()
    v[:, 0] = 448.0                                       # scale 1 in the first block
    rows = [v, v * 2.0 ** -100, v * 2.0 ** 100]
    fi = torch.finfo(DT[dtype])
    ends = torch.zeros(4, C)
    ends[0, :3] = torch.tensor([fi.tiny, fi.tiny * 2 ** -7, fi.tiny / 2])
    ends[1, :3] = torch.tensor([fi.max, fi.min, 1.0])
    ends[2, 3], ends[3, 40] = fi.tiny * 2 ** -7, -0.0
    x = torch.cat(rows + [ends]).to(DT[dtype])
    got = block.pack_rows(x.cuda())
    want = ref.pack(x)
    same_rows8(got, want[0], want[1])
    # below 2^-126 bf16 has no room for all bits of the value: fp32 only
    assert torch.equal(block.unpack_rows(got, torch.float32).cpu().double(), want[2].float().double())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", [96, 99])
def test_rows8_without_numbers(C, dtype):
    inf, nan = math.inf, math.nan
    x = torch.randn(8, C, generator=gen(32))
    x[0, 5], x[1, 7], x[2, 9] = inf, -inf, nan
    x[3], x[4] = -inf, nan
    x[5] = torch.finfo(DT[dtype]).min
    x[6, :32], x[6, 40] = inf, -inf
    x[7, 64:96] = -inf
    x[7, 70] = nan
    x = x.to(DT[dtype])
    codes, exps, values = ref.pack(x)
    got = block.pack_rows(x.cuda())
    same_rows8(got, codes, exps)
    back = block.unpack_rows(got, torch.float32).cpu().double()
    assert torch.equal(torch.isnan(back), torch.isnan(values))
    keep = ~torch.isnan(values)
    assert torch.equal(back[keep], values[keep])
    assert bool((back[3] == -inf).all()) and bool((back[5] == -inf).all())


def test_rows8_shapes():
    """Leading dimensions, sliced ones among them."""
    x = torch.randn(3, 5, 96, generator=gen(33)).cuda()
    p = block.pack_rows(x[:, :, 32:])
    assert p.codes.shape == (3, 5, 64) and p.scales.shape == (3, 5, 2)
    q = block.pack_rows(x[:, :, 32:].reshape(15, 64))
    assert torch.equal(p.codes.view(torch.uint8).view(15, 64), q.codes.view(torch.uint8))


# ---- norm with the residual's addition -------------------------------------

NORM = [
    # R, C, kind, weight, bias, slices of x and residual (extra columns, first column)
    (1, 1, "rms", True, False, None, None),
    (3, 7, "layer", True, True, None, None),
    (5, 33, "rms", False, False, (3, 1), None),
    (70, 64, "layer", True, True, (64, 8), (8, 0)),
    (33, 128, "rms", True, False, None, (128, 128)),
    (9, 136, "layer", False, True, None, None),
    (6, 512, "rms", True, True, (8, 8), None),
    (5, 513, "rms", True, False, None, None),
    (7, 1003, "layer", True, True, None, (2, 1)),
    (4, 1024, "rms", True, False, None, None),
    (3, 2048, "layer", True, True, None, None),
    (3, 2049, "rms", True, False, None, None),
    (5, 2056, "rms", False, False, None, None),
    (2, 4096, "layer", True, True, None, None),
    (2, 5000, "rms", True, True, None, None),
    (2, 8195, "layer", True, False, None, None),
    (2, 8200, "rms", True, False, None, None),
    (2, 16384, "layer", True, True, None, None),
    (1, 16383, "rms", True, True, None, None),
    (2100, 72, "rms", True, False, None, None),
    (600, 2048, "rms", True, False, None, None),
    (0, 64, "rms", True, True, None, None),
]
NORM_IDS = [f"R{c[0]}C{c[1]}{c[2]}" for c in NORM]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def norm_case(c, types, seed):
    R, C, kind, with_w, with_b, cx, cr = c
    g = gen(seed)
    x, res = rn(g, R, C, dtype=DT[types[0]]), rn(g, R, C, dtype=DT[types[1]], std=2.0) + (3.0 if kind == "layer" else 0.0)
    res = res.to(DT[types[1]])
    if cx:
        x = sliced(x, *cx)
    if cr:
        res = sliced(res, *cr)
    return x, res, (1 + 0.1 * rn(g, C)) if with_w else None, rn(g, C) if with_b else None


def check_y(y, n):
    """The 64-bit norm rounded once: half a step (sums in another order move
    the 64-bit value by 2^-40 of it at most)."""
    tol = (half_step(y.dtype) + 2.0 ** -40) * n.abs() + 2.0 ** -40 + 1e-38
    assert bool(((y.cpu().double() - n).abs() <= tol).all())


@pytest.mark.parametrize("types", TYPES, ids=["-".join(t) for t in TYPES])
@pytest.mark.parametrize("c", NORM, ids=NORM_IDS)
def test_add_norm_forward(c, types):
    x, res, w, b = norm_case(c, types, 41)
    R, C, kind = c[:3]
    out = {"h": Guarded((R, C), res.dtype), "y": Guarded((R, C), x.dtype), "y8": Guarded8((R, C)), "h8": Guarded8((R, C))}
    got = block.add_norm_forward(x, res, w, b, eps=1e-3, kind=kind, want=("h", "y", "y8", "h8"), out={n: t.t for n, t in out.items()})
    torch.cuda.synchronize()
    for n, t in out.items():
        t.check(n)
    h = ref.add(x, res)
    assert torch.equal(got["h"].cpu().double(), h)
    n = ref.norm(h, w, b, 1e-3, kind)
    check_y(got["y"], n)
    if R <= 100:
        # a value within 2^-40 of a border between two codes would be open; none is
        same_rows8(got["y8"], *ref.pack(n)[:2], "y8")
        same_rows8(got["h8"], *ref.pack(h)[:2], "h8")
    else:
        again = block.pack_rows(got["h"])
        assert torch.equal(again.codes.view(torch.uint8), got["h8"].codes.view(torch.uint8))
    # each output by itself is the same
    for name in ("h", "y", "y8", "h8"):
        one = block.add_norm_forward(x, res, w, b, eps=1e-3, kind=kind, want=(name,))
        assert [k for k, v in one.items() if v is not None] == [name]
        for u, v in zip(one[name] if isinstance(one[name], tuple) else (one[name],),
                        got[name] if isinstance(got[name], tuple) else (got[name],)):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8)), name


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", [64, 37, 2048])
def test_add_norm_without_residual_and_in_place(C, dtype):
    g = gen(42)
    x, res, w = rn(g, 5, C, dtype=DT[dtype]), rn(g, 5, C, dtype=DT[dtype]), rn(g, C)
    o = block.add_norm_forward(x, None, w, want=("h", "y", "h8"))
    assert torch.equal(o["h"], x)
    check_y(o["y"], ref.norm(ref.add(x, None), w, None, 1e-5, "rms"))
    want = block.add_norm_forward(x, res, w)
    stream = res.clone()
    got = block.add_norm_forward(x, stream, w, out={"h": stream})
    assert got["h"] is stream and torch.equal(stream, want["h"]) and torch.equal(got["y"], want["y"])


def test_add_norm_rows_without_numbers():
    """A row of infinities or NaN stays by itself; a row of zeros has n = bias."""
    g = gen(43)
    x = rn(g, 6, 64)
    x[1, 3], x[2, 5], x[4] = math.inf, math.nan, 0.0
    b = rn(g, 64)
    o = block.add_norm_forward(x, torch.zeros_like(x), None, b, want=("h", "y", "y8"))
    y = o["y"].cpu()
    assert not bool(torch.isfinite(y[2]).any()) and math.isnan(float(y[1, 3]))
    assert torch.equal(y[4], b.cpu())
    assert bool(torch.isfinite(y[[0, 3, 5]]).all())
    same_rows8(block.Rows8(o["y8"].codes[[0, 3, 5]], o["y8"].scales[[0, 3, 5]]),
               *ref.pack(ref.norm(ref.add(x[[0, 3, 5]], None), None, b, 1e-5, "rms"))[:2])


@pytest.mark.parametrize("C", [64, 99, 2048, 9000])
@pytest.mark.parametrize("types", TYPES, ids=["-".join(t) for t in TYPES])
def test_add_norm_ends_of_the_stream(types, C):
    """Streams whose squares pass fp32's range on either side keep their norm
    and its gradients; under an infinity the rms norm of the others is the bias."""
    g = gen(44)
    x, dy, w, b = rn(g, 5, C, dtype=DT[types[0]]), rn(g, 5, C, dtype=DT[types[0]]), rn(g, C), rn(g, C)
    res = torch.zeros(5, C, dtype=DT[types[1]]).cuda()
    x[0], x[1], x[2] = x[0] * 2.0 ** 100, x[1] * 2.0 ** 120, x[2] * 2.0 ** -90
    for kind in ("rms", "layer"):
        o = block.add_norm_forward(x, res, w, b, 0.0, kind, want=("h", "y", "h8"))
        check_y(o["y"], ref.norm(ref.add(x, res), w, b, 0.0, kind))
        got = block.add_norm_backward(o["h"], dy, None, w, b, 0.0, kind)
        want, bound = ref.norm_grad(o["h"].cpu().double(), dy, None, w, 0.0, kind)
        norm_grad_close(got, want, bound, 5, C, DT[types[1]], DT[types[0]])
    x[3, 5] = math.inf
    y = block.add_norm_forward(x, res, w, b)["y"][3].cpu()
    want = b.cpu().to(y.dtype)
    want[5] = math.nan
    assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))


def norm_grad_close(got, want, bound, R, C, stream, rows, name=""):
    # the row's sums: C / 8 elements in sequence, then lanes; dx passes three of them
    close(got["dresidual"], want["dresidual"], bound["dresidual"], 96 + C / 4, name + "dresidual")
    if stream is not rows:
        close(got["dx"], want["dresidual"], bound["dresidual"], 96 + C / 4, name + "dx")
    for n in ("dweight", "dbias"):
        if got[n] is not None:
            close(got[n], want[n], bound[n], 96 + C / 4 + R, name + n)


@pytest.mark.parametrize("types", TYPES, ids=["-".join(t) for t in TYPES])
@pytest.mark.parametrize("c", NORM, ids=NORM_IDS)
def test_add_norm_backward(c, types):
    x, res, w, b = norm_case(c, types, 44)
    R, C, kind = c[:3]
    g = gen(45)
    dy, dh = rn(g, R, C, dtype=DT[types[0]]), rn(g, R, C, dtype=DT[types[1]])
    o = block.add_norm_forward(x, res, w, b, eps=1e-3, kind=kind, want=("h", "h8"))
    for name, src, more in (("h ", o["h"], dh), ("h8 ", o["h8"], dh), ("no dh ", o["h"], None)):
        kw = dict(dh=more, weight=w, bias=b, eps=1e-3, kind=kind)
        out = {"dresidual": Guarded((R, C), res.dtype)}
        if types[0] != types[1]:
            out["dx"] = Guarded((R, C), x.dtype)
        for n, p in (("dweight", w), ("dbias", b)):
            if p is not None:
                out[n] = Guarded((C,), torch.float32)
        got = block.add_norm_backward(src, dy, out={n: t.t for n, t in out.items()}, **kw)
        torch.cuda.synchronize()
        for n, t in out.items():
            t.check(n)
        again = block.add_norm_backward(src, dy, **kw)
        assert all(torch.equal(got[n], again[n]) for n in got if got[n] is not None)
        assert got["dx"].dtype == x.dtype and got["dresidual"].dtype == res.dtype
        values = block.unpack_rows(src, torch.float32).cpu().double() if isinstance(src, tuple) else src.cpu().double()
        want, bound = ref.norm_grad(values, dy, more, w, 1e-3, kind)
        norm_grad_close(got, want, bound, R, C, res.dtype, x.dtype, name)


def test_add_norm_backward_in_place():
    g = gen(46)
    h, dy, dh, w = rn(g, 9, 136), rn(g, 9, 136), rn(g, 9, 136), rn(g, 136)
    want = block.add_norm_backward(h, dy, dh, w)
    got = block.add_norm_backward(h, dy, dh, w, out={"dresidual": dh})
    assert got["dresidual"] is dh and torch.equal(dh, want["dresidual"]) and torch.equal(got["dweight"], want["dweight"])


# ---- gated linear recurrence -----------------------------------------------

LENGTHS = [0, 1, 2, 17, 0, 16, 64, 15, 270, 0, 513]     # packed: five rows before, seven behind


def packed():
    offs = [5]
    for n in LENGTHS:
        offs.append(offs[-1] + n)
    return torch.tensor(offs, dtype=torch.int64).cuda(), offs[-1] + 7


GLR = [
    # B, T, C, packed, init, slices (extra columns, first column) of x and of the gates, algo
    (1, 1, 1, False, False, None, None, "auto"),
    (2, 2, 3, False, True, None, (2, 1), "auto"),
    (1, 15, 64, False, True, None, None, "auto"),
    (3, 16, 66, False, True, (66, 66), None, "staged"),
    (2, 17, 65, False, False, (1, 0), None, "staged"),
    (1, 33, 40, False, True, None, (40, 0), "segmented"),
    (2, 129, 34, False, True, None, None, "segmented"),
    (1, 257, 130, False, True, None, None, "auto"),
    (2, 511, 32, False, False, None, (2, 2), "staged"),
    (1, 700, 33, False, True, None, None, "segmented"),
    (1, 1500, 20, False, True, None, None, "segmented"),
    (1, 2100, 70, False, True, None, None, "auto"),
    (200, 20, 64, False, True, None, None, "auto"),        # lanes along 64 channels: enough workgroups
    (100, 40, 96, False, True, None, None, "auto"),
    (0, 0, 34, True, True, None, None, "auto"),
    (0, 0, 64, True, False, (2, 2), None, "staged"),
    (0, 0, 66, True, True, None, (6, 4), "segmented"),
    (0, 0, 7, True, True, None, None, "segmented"),
    (0, 0, 65, True, False, (3, 2), None, "staged"),
    (3, 0, 8, False, True, None, None, "auto"),
]
GLR_IDS = [f"B{c[0]}T{c[1]}C{c[2]}{'p' if c[3] else ''}-{c[7]}" for c in GLR]


def glr_case(c, dtype, seed):
    B, T, C, is_packed, init, cx, cg, algo = c
    g = gen(seed)
    offsets, lead = None, (B, T)
    if is_packed:
        offsets, T = packed()
        B, lead = len(LENGTHS), (T,)
    rows = [rn(g, *lead, C, dtype=DT[dtype]).clamp(-5, 5) for _ in range(3)]
    for k, cut in enumerate((cx, cg, cg)):
        if cut:
            rows[k] = sliced(rows[k], *cut)
    A = -(torch.rand(C, generator=g) * 0.95 + 0.005).cuda()
    if C > 2:
        A[1] = 0.0                                          # a = 1: the state stays
    h0 = rn(g, B, C) if init else None
    return rows, A, h0, offsets, B, T, algo


def cut_of(offsets):
    return slice(None) if offsets is None else slice(int(offsets[0]), int(offsets[-1]))


def untouched(t, offsets):
    s = torch.tensor(SENT, dtype=t.dtype, device=t.device)
    return bool((t[:int(offsets[0])] == s).all()) and bool((t[int(offsets[-1]):] == s).all())


def chunk_rows(offsets, B, T):
    """(sequence, its 16-token piece) -> row of h_chunks."""
    if offsets is None:
        return lambda s, j: s * -(-T // 16) + j
    o = [int(v) for v in offsets]
    return lambda s, j: o[s] // 16 + s + j


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", GLR, ids=GLR_IDS)
def test_glr_forward(c, dtype):
    (x, r, i), A, h0, offsets, B, T, algo = glr_case(c, dtype, 51)
    C = A.shape[0]
    nck = block.glr_chunk_count(B, T, offsets is not None)
    y, ho, ck = Guarded(x.shape, x.dtype), Guarded((B, C), torch.float32), Guarded((nck, C), torch.float32)
    y.t.fill_(SENT), ck.t.fill_(SENT)
    got, h, chunks = block.glr_forward(x, r, i, A, h0, offsets, out=y.t, h_out=ho.t, chunk_states=ck.t, algo=algo)
    torch.cuda.synchronize()
    y.check("y"), ho.check("h"), ck.check("chunks")
    wy, by, wh, bh, marks = ref.glr(x, r, i, A, h0, offsets)
    cut = cut_of(offsets)
    if offsets is not None:
        assert untouched(got, offsets)
    close(got[cut], wy[cut], by[cut], 64, "y")
    close(h, wh, bh, 64, "h")
    at, used = chunk_rows(offsets, B, T), set()
    for s, rec in enumerate(marks):
        for j, (state, bound) in enumerate(rec):
            used.add(at(s, j))
            close(chunks[at(s, j)], state, bound, 64, f"state {s} {j}")
    rest = [k for k in range(nck) if k not in used]
    assert bool((chunks[rest] == SENT).all())
    # the same without the extras, and in place on the state
    again = block.glr_forward(x, r, i, A, h0, offsets, algo=algo)
    assert torch.equal(again[0][cut], got[cut]) and torch.equal(again[1], h)
    if h0 is not None:
        st = h0.clone()
        block.glr_forward(x, r, i, A, st, offsets, h_out=st, algo=algo)
        assert torch.equal(st, h)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", GLR, ids=GLR_IDS)
def test_glr_checkpoint(c, dtype):
    """The rows in 8 bits are those of pack_rows; results stay what they are."""
    (x, r, i), A, h0, offsets, B, T, algo = glr_case(c, dtype, 52)
    saved = [Guarded8(tuple(x.shape)) for _ in range(3)]
    for s in saved:
        for t in s.t:
            t.view(torch.uint8).fill_(0x5A)
    y, h, ck, got = block.glr_forward(x, r, i, A, h0, offsets, checkpoint=[s.t for s in saved], algo=algo)
    torch.cuda.synchronize()
    plain = block.glr_forward(x, r, i, A, h0, offsets, chunk_states=True, algo=algo)
    cut = cut_of(offsets)
    assert torch.equal(y[cut], plain[0][cut]) and torch.equal(h, plain[1])
    for s, p, t in zip(saved, got, (x, r, i)):
        s.check("rows8")
        want = block.pack_rows(t)
        for u, v in zip(p, want):
            u, v = u.view(torch.uint8), v.view(torch.uint8)
            assert torch.equal(u[cut], v[cut])
            if offsets is not None:
                assert bool((u[:cut.start] == 0x5A).all()) and bool((u[cut.stop:] == 0x5A).all())


def check_glr_grads(got, want, bound, cut, tokens):
    for n in ("dx", "dr", "di"):
        close(got[n][cut], want[n][cut], bound[n][cut], 192, n)
    close(got["dA"], want["dA"], bound["dA"], 192 + tokens, "dA")
    if got["dh0"] is not None:
        close(got["dh0"], want["dh0"], bound["dh0"], 192, "dh0")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", GLR, ids=GLR_IDS)
def test_glr_backward(c, dtype):
    (x, r, i), A, h0, offsets, B, T, algo = glr_case(c, dtype, 53)
    C, g = A.shape[0], gen(54)
    dy, dh = rn(g, *x.shape, dtype=x.dtype), rn(g, B, C) if c[4] else None
    _, _, ck = block.glr_forward(x, r, i, A, h0, offsets, chunk_states=True, algo=algo)
    out = {n: Guarded(x.shape, x.dtype) for n in ("dx", "dr", "di")}
    out["dA"], out["dh0"] = Guarded((C,), torch.float32), Guarded((B, C), torch.float32)
    for t in out.values():
        t.t.fill_(SENT)
    kw = dict(offsets=offsets, dh_out=dh, algo=algo)
    got = block.glr_backward(x, r, i, A, dy, ck, out={n: t.t for n, t in out.items()}, **kw)
    torch.cuda.synchronize()
    for n, t in out.items():
        t.check(n)
    cut = cut_of(offsets)
    if offsets is not None:
        assert all(untouched(got[n], offsets) for n in ("dx", "dr", "di"))
    again = block.glr_backward(x, r, i, A, dy, ck, **kw)
    for n in got:
        part = cut if n in ("dx", "dr", "di") else slice(None)
        assert torch.equal(got[n][part], again[n][part]), n
    want, bound = ref.glr_grad(x, r, i, A, dy, h0, offsets, dh)
    check_glr_grads(got, want, bound, cut, x.numel() // C)
    if dh is not None:
        st = dh.clone()
        block.glr_backward(x, r, i, A, dy, ck, offsets=offsets, dh_out=st, algo=algo, out={"dh0": st})
        assert torch.equal(st, got["dh0"])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("c", GLR, ids=GLR_IDS)
def test_glr_backward_from_8_bits(c, dtype):
    (x, r, i), A, h0, offsets, B, T, algo = glr_case(c, dtype, 55)
    C, g = A.shape[0], gen(56)
    dy, dh = rn(g, *x.shape, dtype=x.dtype), rn(g, B, C) if c[4] else None
    _, _, ck, saved = block.glr_forward(x, r, i, A, h0, offsets, checkpoint=True, algo=algo)
    got = block.glr_backward(*saved, A, dy, ck, offsets=offsets, dh_out=dh, algo=algo)
    values = [block.unpack_rows(p, torch.float32) for p in saved]
    at = chunk_rows(offsets, B, T)
    seqs = ref.sequences(x.shape, offsets)
    marks = ref.glr(x, r, i, A, h0, offsets)[4]
    # (state, its magnitude): the recorded states are exact here, an error in them is none of the gradients'
    starts = [[(ck[at(s, j)].cpu().double(), ck[at(s, j)].cpu().double().abs()) for j in range(len(marks[s]))] for s in range(len(seqs))]
    want, bound = ref.glr_grad(*values, A, dy, h0, offsets, dh, starts)
    check_glr_grads(got, want, bound, cut_of(offsets), x.numel() // C)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", [33, 64])
@pytest.mark.parametrize("mask", ["inf", "lowest"])
def test_glr_masked_tokens(mask, C, dtype):
    """A masked token leaves the state as it is, whatever it holds, also from
    rows in 8 bits; a sequence that is masked whole hands its state on."""
    g = gen(57)
    B, T = 3, 300
    x, r, i, dy = (rn(g, B, T, C, dtype=DT[dtype]) for _ in range(4))
    A, h0, dh = -torch.rand(C, generator=g).cuda(), rn(g, B, C), rn(g, B, C)
    off = torch.zeros(B, T, dtype=torch.bool)
    off[0, 250:], off[1, [0, 1, 15, 16, 17, 255, 256, 299]], off[2] = True, True, True
    r[off.cuda()] = -math.inf if mask == "inf" else torch.finfo(DT[dtype]).min
    x[0, 260], x[1, 16], i[1, 17], x[2, 5], i[2, 6] = math.nan, math.inf, math.nan, -math.inf, math.inf
    y, h, ck, saved = block.glr_forward(x, r, i, A, h0, checkpoint=True)
    wy, by, wh, bh, _ = ref.glr(x, r, i, A, h0)
    close(y, wy, by, 64, "y")
    close(h, wh, bh, 64, "h")
    assert torch.equal(h[2], h0[2]) and bool((y[2] == h0[2].to(y.dtype)).all())
    got = block.glr_backward(x, r, i, A, dy, ck, dh_out=dh)
    want, bound = ref.glr_grad(x, r, i, A, dy, h0, None, dh)
    check_glr_grads(got, want, bound, slice(None), B * T)
    eight = block.glr_backward(*saved, A, dy, ck, dh_out=dh)
    for gr in (got, eight):
        assert all(bool((gr[n][off.cuda()] == 0).all()) for n in ("dx", "dr", "di"))
        assert all(bool(torch.isfinite(gr[n]).all()) for n in gr)


def test_glr_ends_of_the_parameters():
    """A = -inf empties the state in every open token; a NaN stays a NaN."""
    g = gen(58)
    x, r, i = (rn(g, 2, 40, 6) for _ in range(3))
    A = torch.tensor([-math.inf, math.nan, -1e30, 0.0, -100.0, -1e-30]).cuda()
    r[:, 7] = -math.inf
    y, h = block.glr_forward(x, r, i, A)
    si = torch.sigmoid(i.cpu().double())
    want = si * x.cpu().double()
    keep = [t for t in range(40) if t != 7]
    for c in (0, 2):
        close(y[:, keep, c], want[:, keep, c], want[:, keep, c].abs(), 64)
        assert torch.equal(y[:, 7, c], y[:, 6, c])
    assert bool(torch.isnan(y[..., 1]).all()) and not bool(y[..., 3].any())
    wy, by, _, _, _ = ref.glr(x[..., 4:], r[..., 4:], i[..., 4:], A[4:])
    # exponents of up to 100 multiply the roundings of s(r)
    close(y[..., 4:], wy, by, 64 * 100)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("N,C,cut", [(1, 1, None), (3, 64, (64, 0)), (5, 37, (2, 1)), (130, 260, None), (0, 8, None), (2, 4100, None)])
def test_glr_step(N, C, cut, dtype):
    g = gen(59)
    x, r, i = (rn(g, N, C, dtype=DT[dtype]).clamp(-5, 5) for _ in range(3))
    if cut:
        x, r = sliced(x, *cut), sliced(r, *cut)
    A, st = -torch.rand(C, generator=g).cuda(), rn(g, N, C)
    if N:
        r[0] = -math.inf
        x[0, 0] = math.nan
    wy, by, wh, bh, _ = ref.glr(x[:, None], r[:, None], i[:, None], A, st)
    y, s = Guarded((N, C), x.dtype), Guarded((N, C), torch.float32)
    s.t.copy_(st)
    block.glr_step(s.t, x, r, i, A, out=y.t)
    torch.cuda.synchronize()
    y.check("y"), s.check("state")
    close(y.t, wy[:, 0], by[:, 0], 64, "y")
    close(s.t, wh, bh, 64, "state")


def test_glr_prompt_then_tokens():
    """A prompt, its continuation, and single tokens give one sequence."""
    g = gen(60)
    x, r, i = (rn(g, 2, 301, 70) for _ in range(3))
    A = -torch.rand(70, generator=g).cuda()
    y, h = block.glr_forward(x, r, i, A)
    parts = lambda a, b: [t[:, a:b] for t in (x, r, i)]  # noqa: E731
    y1, st = block.glr_forward(*(t.contiguous() for t in parts(0, 150)), A)
    y2, st = block.glr_forward(*(t.contiguous() for t in parts(150, 290)), A, st)
    ys = [y1, y2] + [block.glr_step(st, x[:, t], r[:, t], i[:, t], A)[:, None] for t in range(290, 301)]
    _, by, _, bh, _ = ref.glr(x, r, i, A)
    close(torch.cat(ys, 1), y.cpu().double(), by, 64)
    close(st, h.cpu().double(), bh, 64)


# ---- streams, graphs, a block of them --------------------------------------

def test_two_at_once():
    """Calls on two streams with buffers of their own do not disturb one another."""
    g = gen(61)
    sets = [[rn(g, 4, 600, 128, dtype=torch.bfloat16) for _ in range(3)] for _ in range(2)]
    A, res = -torch.rand(128, generator=g).cuda(), rn(g, 4, 600, 128, dtype=torch.bfloat16)
    w = rn(g, 128)

    def work(s):
        o = block.add_norm_forward(s[0], res, w, want=("h", "y", "h8"))
        y, _, ck, saved = block.glr_forward(o["y"], s[1], s[2], A, checkpoint=True, algo="segmented")
        gr = block.glr_backward(*saved, A, y, ck, algo="segmented")
        nb = block.add_norm_backward(o["h8"], gr["dx"], None, w)
        return [y, gr["dr"], gr["di"], gr["dA"], nb["dx"], nb["dweight"]]

    want = [work(s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[k].append(work(sets[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[k]))


def test_captured_graph():
    """A training step of a block, captured and replayed with new inputs."""
    g = gen(62)
    B, T, C = 2, 300, 128
    x, r, i, dy = (rn(g, B, T, C, dtype=torch.bfloat16) for _ in range(4))
    res, w, A = rn(g, B, T, C), rn(g, C), -torch.rand(C, generator=g).cuda()

    def step():
        o = block.add_norm_forward(x, res, w, want=("h", "y", "y8", "h8"))
        y, h, ck, saved = block.glr_forward(o["y"], r, i, A, checkpoint=True, algo="segmented")
        gr = block.glr_backward(*saved, A, dy, ck, algo="segmented")
        nb = block.add_norm_backward(o["h8"], gr["dx"], res, w)
        return [o["h"], o["y8"].codes.view(torch.uint8), y, h, gr["dr"], gr["di"], gr["dA"], nb["dresidual"], nb["dx"], nb["dweight"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for n in range(4):
        for t in (x, r, i, dy):
            t.copy_(rn(g, B, T, C, dtype=torch.bfloat16))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), n


@pytest.mark.parametrize("eight", [False, True])
def test_training_step_of_a_block(eight):
    """h = x + residual, n = rms(h) w, (z, r, i) = n W, y = recurrence, back to
    the residual: gradients against automatic differentiation of the same block
    in 64 bits; from rows in 8 bits they are near them."""
    g = gen(63)
    B, T, C = 2, 150, 64
    x, res = rn(g, B, T, C), rn(g, B, T, C)
    w, W, A, dy = 1 + 0.1 * rn(g, C), rn(g, C, 3 * C, std=C ** -0.5), -torch.rand(C, generator=g).cuda() - 0.01, rn(g, B, T, C)
    o = block.add_norm_forward(x, res, w, want=("h", "y", "h8"))
    p = o["y"] @ W
    z, r, i = p[..., :C], p[..., C:2 * C], p[..., 2 * C:]
    y, _, ck, saved = block.glr_forward(z, r, i, A, checkpoint=True)
    gr = block.glr_backward(*(saved if eight else (z, r, i)), A, dy, ck)
    dp = torch.cat([gr["dx"], gr["dr"], gr["di"]], -1)
    nb = block.add_norm_backward(o["h8"] if eight else o["h"], dp @ W.t(), dy, w)

    leaves = [t.detach().cpu().double().requires_grad_() for t in (x, w, W, A)]
    lx, lw, lW, lA = leaves
    h = lx + res.cpu().double()
    n = h * (h.square().mean(-1, keepdim=True) + 1e-5) ** -0.5 * lw
    lz, lr, li = (n @ lW).split(C, -1)
    u = lA * torch.sigmoid(lr)
    a, b = torch.exp(u), torch.sqrt(-torch.expm1(2 * u)) * torch.sigmoid(li) * lz
    st, out = torch.zeros(B, C, dtype=torch.float64), []
    for t in range(T):
        st = a[:, t] * st + b[:, t]
        out.append(st)
    d = dy.cpu().double()
    want = torch.autograd.grad((torch.stack(out, 1) * d).sum() + (h * d).sum(), leaves)
    got = (nb["dx"], nb["dweight"], torch.einsum("btc,btd->cd", o["y"].cpu().double(), dp.cpu().double()), gr["dA"])
    for k, (u, v) in enumerate(zip(got, want)):
        err = float((u.cpu().double() - v).norm() / v.norm())
        # fp32 throughout: some hundred roundings of 2^-24 over 150 tokens' memory.  A code is off by 2^-4 of its value
        # at most, 2.6 % on average; a gradient has up to four such factors.
        assert err < (0.1 if eight else 1e-4), (k, err)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("is_packed", [False, True])
def test_glr_long_chains(is_packed, dtype):
    """Tiles chained over dozens of others, alike in every run; also in one pass."""
    g = gen(64)
    C, T = 70, 6000
    offsets = torch.tensor([0, 0, 3, 5403, 5403, 5404, 6000, 6000]).cuda() if is_packed else None
    B, lead = (7, (T,)) if is_packed else (1, (1, T))
    x, r, i, dy = (rn(g, *lead, C, dtype=DT[dtype]).clamp(-5, 5) for _ in range(4))
    A, h0, dh = -torch.rand(C, generator=g).cuda(), rn(g, B, C), rn(g, B, C)
    A[0] = 0.0
    wy, by, wh, bh, _ = ref.glr(x, r, i, A, h0, offsets)
    want, bound = ref.glr_grad(x, r, i, A, dy, h0, offsets, dh)
    for algo in ("segmented", "staged"):
        first = None
        for _ in range(4):
            y, h, ck = block.glr_forward(x, r, i, A, h0, offsets, chunk_states=True, algo=algo)
            got = block.glr_backward(x, r, i, A, dy, ck, offsets, dh, algo=algo)
            now = [y, h, *got.values()]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
            first = now
        close(y, wy, by, 64, "y")
        close(h, wh, bh, 64, "h")
        check_glr_grads(got, want, bound, slice(None), T)


def test_glr_of_the_training_shape():
    """8 x 4096 x 2048: the channels are independent, a few of them are checked."""
    g = torch.Generator(device="cuda").manual_seed(65)
    B, T, C = 8, 4096, 2048
    x, r, i, dy = (torch.randn(B, T, C, device="cuda", generator=g).to(torch.bfloat16) for _ in range(4))
    A = -torch.rand(C, device="cuda", generator=g)
    pick = torch.tensor([0, 63, 64, 2047]).cuda()
    few = [t[..., pick].contiguous() for t in (x, r, i)]
    wy, by, wh, bh, _ = ref.glr(*few, A[pick])
    want, bound = ref.glr_grad(*few, A[pick], dy[..., pick], None, None, None)
    y, h, ck, saved = block.glr_forward(x, r, i, A, checkpoint=True)
    plain, last, ck1 = block.glr_forward(x, r, i, A, chunk_states=True)
    for a, b in ((y, h), (plain, last)):
        close(a[..., pick], wy, by, 64, "y")
        close(b[..., pick], wh, bh, 64, "h")
    for p, t in zip(saved, (x, r, i)):
        assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(p, block.pack_rows(t)))
    for states in (ck, ck1):
        got = block.glr_backward(x, r, i, A, dy, states)
        got = {n: t[..., pick] for n, t in got.items()}
        check_glr_grads(got, want, bound, slice(None), B * T)


def test_workspaces_of_the_callers_own():
    """One workspace for calls in turn, larger than needed and full of anything."""
    g = gen(66)
    x, r, i, dy = (rn(g, 2, 1500, 66, dtype=torch.bfloat16) for _ in range(4))
    A, w = -torch.rand(66, generator=g).cuda(), rn(g, 66)
    y, h, ck = block.glr_forward(x, r, i, A, chunk_states=True, algo="segmented")
    want = block.glr_backward(x, r, i, A, dy, ck, algo="segmented")
    nw = block.add_norm_backward(x, dy, None, w)
    space = torch.full((1 << 22,), 0xC0, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        y1, h1, ck1 = block.glr_forward(x, r, i, A, chunk_states=True, algo="segmented", workspace=space)
        got = block.glr_backward(x, r, i, A, dy, ck1, algo="segmented", workspace=space)
        nb = block.add_norm_backward(x, dy, None, w, workspace=space)
        assert torch.equal(y, y1) and torch.equal(h, h1) and torch.equal(ck, ck1)
        assert all(torch.equal(got[n], want[n]) for n in want)
        assert all(torch.equal(nb[n], nw[n]) for n in ("dx", "dweight"))


@pytest.mark.parametrize("algo", ["staged", "segmented"])
def test_glr_bad_offsets_stay_inside(algo):
    """Offsets out of range or descending are clamped on the device: the calls
    return and write only their outputs' rows."""
    g = gen(67)
    T, C = 600, 34
    x, r, i, dy = (rn(g, T, C, dtype=torch.bfloat16) for _ in range(4))
    A, nck = -torch.rand(C, generator=g).cuda(), block.glr_chunk_count(2, T, True)
    for offs in ([-5, 300, 900], [400, 10, 500], [0, 1 << 60, -(1 << 60)], [600, 600, 600], [700, 700, 700], [0, 599, 300]):
        o = torch.tensor(offs, dtype=torch.int64).cuda()
        y, h, ck = Guarded(x.shape, x.dtype), Guarded((2, C), torch.float32), Guarded((nck, C), torch.float32)
        saved = [Guarded8((T, C)) for _ in range(3)]
        block.glr_forward(x, r, i, A, None, o, out=y.t, h_out=h.t, chunk_states=ck.t, checkpoint=[s.t for s in saved], algo=algo)
        grads = {n: Guarded(x.shape, x.dtype) for n in ("dx", "dr", "di")}
        grads.update(dA=Guarded((C,), torch.float32), dh0=Guarded((2, C), torch.float32))
        block.glr_backward(x, r, i, A, dy, torch.zeros_like(ck.t), o, algo=algo, out={n: t.t for n, t in grads.items()})
        torch.cuda.synchronize()
        for n, b in (("y", y), ("h", h), ("chunks", ck), *enumerate(saved), *grads.items()):
            b.check(n)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_far_apart():
    """Rows whose byte offsets pass 32 bits: slices of wide rows against their copies."""
    g = torch.Generator(device="cuda").manual_seed(68)
    R, C, wide = 40001, 70, 1 << 16
    far = torch.empty(R, wide, dtype=torch.bfloat16, device="cuda")[:, 6:6 + C]       # 5.2 GB
    far.copy_(torch.randn(R, C, device="cuda", generator=g))
    near, A, w = far.contiguous(), -torch.rand(C, device="cuda", generator=g), torch.rand(C, device="cuda", generator=g)
    assert all(same(u, v) for u, v in zip(block.pack_rows(far), block.pack_rows(near)))
    got, want = (block.add_norm_forward(t, t, w, want=("h", "y", "y8")) for t in (far, near))
    assert same(got["h"], want["h"]) and same(got["y"], want["y"]) and same(got["y8"].codes, want["y8"].codes)
    for algo in ("staged", "segmented"):
        fwd = [block.glr_forward(t[None], t[None], t[None], A, checkpoint=True, algo=algo) for t in (far, near)]
        assert all(same(u, v) for u, v in zip(fwd[0][:3], fwd[1][:3]))
        assert all(same(u, v) for p, q in zip(fwd[0][3], fwd[1][3]) for u, v in zip(p, q))
        grad = [block.glr_backward(t[None], t[None], t[None], A, near[None], f[2], algo=algo) for t, f in zip((far, near), fwd)]
        assert all(same(grad[0][n], grad[1][n]) for n in grad[0])
    st = [torch.zeros(R, C, device="cuda") for _ in range(2)]
    y = [block.glr_step(s, t, t, t, A) for s, t in zip(st, (far, near))]
    assert same(*y) and same(*st)


def test_arrays_past_4_gib():
    """Dense arrays of more than 2^32 elements: their last rows against the same rows by themselves."""
    g = torch.Generator(device="cuda").manual_seed(69)
    R, C, tail = (1 << 22) + 35, 1024, 8192
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)        # 8.6 GB
    A, w = -torch.rand(C, device="cuda", generator=g) - 0.01, torch.rand(C, device="cuda", generator=g)
    last = x[-tail:].contiguous()
    p, q = block.pack_rows(x), block.pack_rows(last)
    assert same(p.codes[-tail:], q.codes) and same(p.scales[-tail:], q.scales)
    back = block.unpack_rows(p)
    assert same(back[-tail:], block.unpack_rows(q))
    del back, p
    o, part = block.add_norm_forward(x, x, w, want=("h", "y8")), block.add_norm_forward(last, last, w, want=("h", "y8"))
    assert same(o["h"][-tail:], part["h"]) and same(o["y8"].codes[-tail:], part["y8"].codes)
    dx = block.add_norm_backward(o["h"], x, None, w)["dx"]
    assert same(dx[-tail:], block.add_norm_backward(part["h"], last, None, w)["dx"])
    del o, dx
    cut = R // 16 * 16 - tail                                    # of a recorded state
    rows = R - cut
    y, h, ck = block.glr_forward(x[None], x[None], x[None], A, chunk_states=True)
    few = [x[cut:, :6].contiguous()[None]] * 3
    start = ck[cut // 16, :6][None].contiguous()
    wy, by, wh, bh, _ = ref.glr(*few, A[:6], start)
    close(y[:, cut:, :6], wy, by, 64, "y")
    close(h[:, :6], wh, bh, 64, "h")
    got = block.glr_backward(x[None], x[None], x[None], A, x[None], ck)
    want, bound = ref.glr_grad(*few, A[:6], few[0], start, None, None)
    for n in ("dx", "dr", "di"):
        close(got[n][:, cut:, :6], want[n], bound[n], 192, n)
    assert rows > tail


def test_gradients_of_nothing():
    z = torch.zeros(0, 5, 34, device="cuda")
    A = -torch.ones(34, device="cuda")
    got = block.glr_backward(z, z, z, A, z, torch.zeros(0, 34, device="cuda"))
    assert torch.equal(got["dA"], torch.zeros_like(A)) and got["dx"].shape == z.shape and got["dh0"].shape == (0, 34)
    e = torch.zeros(3, 0, 34, device="cuda")
    h = torch.randn(3, 34, device="cuda")
    got = block.glr_backward(e, e, e, A, e, torch.zeros(0, 34, device="cuda"), dh_out=h)
    assert torch.equal(got["dA"], torch.zeros_like(A)) and torch.equal(got["dh0"], h)
