"""GPU tests of the block operators at calls their documentation allows and
tests/test_gpu_block.py does not make, against the same 64-bit implementation
and with its tolerances."""
import math

import pytest
import torch

from gated_delta_rule_86_amd import block
from tests import block_reference as ref
from tests.layer_reference import close
from tests.test_gpu_block import check_glr_grads
from tests.test_gpu_layer import DT, gen, rn

pytestmark = pytest.mark.gpu


def bits(t):
    """Codes as bytes, every NaN alike."""
    u = t.view(torch.uint8)
    return torch.where(u & 0x7F == 0x7F, torch.full_like(u, 0x7F), u) if t.dtype is block.CODES else u


def same_rows8(p, q, name):
    assert torch.equal(p.scales.view(torch.uint8), q.scales.view(torch.uint8)), name
    assert torch.equal(bits(p.codes), bits(q.codes)), name


# ---- recurrence: checkpoints whose last block of columns is a part of one ---

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", [2, 20, 62, 66, 72, 80, 88, 94, 104, 2056])
def test_checkpoints_of_rows_without_numbers(C, dtype):
    """Masks of -inf that begin at each of 32 positions, single masked tokens,
    infinities in the last block of columns alone: the rows pack_rows forms."""
    g = gen(71)
    B, T, last = 32, 300, (C - 1) // 32 * 32
    x, r, i = (rn(g, B, T, C, dtype=DT[dtype]) for _ in range(3))
    for b in range(B):
        r[b, 32 + b:64] = -math.inf
        r[b, 256 + b:] = -math.inf
        x[b, 64 + b] = math.inf
        x[b, 256 + b, last:] = -math.inf
        i[b, 96 + b:128, last:] = -math.inf
        i[b, 160 + b] = math.nan
        i[b, 256 + b, C - 1] = math.inf
    A = -torch.rand(C, generator=g).cuda()
    want = [block.pack_rows(t) for t in (x, r, i)]
    for algo in ("staged", "segmented"):
        saved = block.glr_forward(x, r, i, A, checkpoint=True, algo=algo)[3]
        for n, p, q in zip("xri", saved, want):
            same_rows8(p, q, f"{algo} {n}8")


@pytest.mark.parametrize("C,dtype", [(20, "bf16"), (66, "bf16"), (72, "bf16"), (80, "bf16"), (94, "bf16"), (104, "bf16"), (66, "f32"), (104, "f32")])
def test_gradients_from_8_bits_of_masked_tokens(C, dtype):
    """Values at open tokens too: against the gradients at what the codes stand
    for, from the recorded states.  Whole rows are masked, and at C = 104 the last
    block of columns alone."""
    g = gen(72)
    starts = (17, 20, 24, 26, 28, 29, 30, 31)
    B, T, first = len(starts), 300, 96 if C == 104 else 0
    x, r, i = (rn(g, B, T, C, dtype=DT[dtype]).clamp(-5, 5) for _ in range(3))
    dy, h0, dh = rn(g, B, T, C, dtype=DT[dtype]), rn(g, B, C), rn(g, B, C)
    A = -torch.rand(C, generator=g).cuda()
    off = torch.zeros(B, T, C, dtype=torch.bool)
    for b, s in enumerate(starts):
        off[b, 32 + s:64, first:], off[b, 256 + s:, first:], off[b, [3, 96 + s], first:] = True, True, True
    off = off.cuda()
    r[off] = -math.inf
    # what masked tokens hold is not used
    x[0, 32 + 17, first:], x[1, 290, first:], i[2, 280, first:], i[3, 3, first:] = math.nan, math.inf, -math.inf, math.nan
    for algo in ("staged", "segmented"):
        _, _, ck, saved = block.glr_forward(x, r, i, A, h0, checkpoint=True, algo=algo)
        got = block.glr_backward(*saved, A, dy, ck, dh_out=dh, algo=algo)
        values = [block.unpack_rows(p, torch.float32) for p in saved]
        assert bool((values[1][off] == -math.inf).all())
        pieces = -(-T // 16)
        states = [[(s, s.abs()) for s in ck[b * pieces:(b + 1) * pieces].cpu().double()] for b in range(B)]
        want, bound = ref.glr_grad(*values, A, dy, h0, None, dh, states)
        check_glr_grads(got, want, bound, slice(None), B * T)
        assert all(bool((got[n][off] == 0).all()) for n in ("dx", "dr", "di"))


# ---- recurrence: gates far from 1/2 ----------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("C", [64, 33])
@pytest.mark.parametrize("eight", [False, True])
def test_gradients_of_open_and_closed_gates(eight, C, dtype):
    """Logits of -24 to 24: the slope s (1 - s) keeps its digits where 1 - s
    cancels.  A logit of l is 2 l + 5 roundings in its logistic and in one less it
    (the exponent's product, then as for the logits of 5 that 192 stands for): 4
    factors of a gradient, 19 more units of l, 2 roundings each, 152 more."""
    g = gen(73)
    B, T = 2, 300
    x, dy = rn(g, B, T, C, dtype=DT[dtype]), rn(g, B, T, C, dtype=DT[dtype])
    r, i = ((torch.rand(B, T, C, generator=g) * 48 - 24).to(DT[dtype]).cuda() for _ in range(2))
    A, h0, dh = -torch.rand(C, generator=g).cuda(), rn(g, B, C), rn(g, B, C)
    for algo in ("staged", "segmented"):
        _, _, ck, saved = block.glr_forward(x, r, i, A, h0, checkpoint=True, algo=algo)
        got = block.glr_backward(*(saved if eight else (x, r, i)), A, dy, ck, dh_out=dh, algo=algo)
        values = [block.unpack_rows(p, torch.float32) for p in saved] if eight else [x, r, i]
        states = [[(s, s.abs()) for s in ck[b * 19:(b + 1) * 19].cpu().double()] for b in range(B)] if eight else None
        want, bound = ref.glr_grad(*values, A, dy, h0, None, dh, states)
        sr, si = (torch.sigmoid(-t.cpu().double()) for t in values[1:])          # 1 - s
        for n, slope in (("dx", 1), ("dr", sr), ("di", si)):
            close(got[n], want[n], bound[n] * slope, 192 + 152, f"{algo} {n}")
        close(got["dA"], want["dA"], bound["dA"], 192 + 152 + B * T, "dA")
        close(got["dh0"], want["dh0"], bound["dh0"], 192 + 152, "dh0")


@pytest.mark.parametrize("dtype", list(DT))
def test_gradients_of_gates_at_their_ends(dtype):
    """Logits of +-inf, of the types' ends and past the exponential's range:
    finite gradients, 0 (below every normal number) by the logit; a NaN in r or
    i of an open token stays one, and only where it is."""
    g = gen(74)
    x, dy = rn(g, 2, 40, 8, dtype=DT[dtype]), rn(g, 2, 40, 8, dtype=DT[dtype])
    r, i = rn(g, 2, 40, 8, dtype=DT[dtype]), rn(g, 2, 40, 8, dtype=DT[dtype])
    fi = torch.finfo(DT[dtype])
    ends = torch.tensor([math.inf, -math.inf, fi.max, fi.min, 200.0, -200.0, 87.5, 95.0]).to(DT[dtype]).cuda()
    r[0, 4], r[1, 9], i[0, 20], i[1, 4] = ends, ends, ends, ends
    A = -torch.rand(8, generator=g).cuda() - 0.1
    _, _, ck = block.glr_forward(x, r, i, A, chunk_states=True)
    got = block.glr_backward(x, r, i, A, dy, ck)
    want, bound = ref.glr_grad(x, r, i, A, dy)
    for n in ("dx", "dr", "di", "dA", "dh0"):
        close(got[n], want[n], bound[n], 192 + 152, n)
    assert bool((got["dr"][0, 4].abs() < 1e-34).all()) and bool((got["di"][0, 20].abs() < 1e-34).all())
    r[0, 30, 2], i[1, 30, 3] = math.nan, math.nan
    got = block.glr_backward(x, r, i, A, dy, ck)
    assert bool(torch.isnan(got["dr"][0, 30, 2])) and bool(torch.isnan(got["di"][1, 30, 3]))
    others = [c for c in range(8) if c != 2]
    assert bool(torch.isfinite(got["dr"][0][:, others]).all()) and bool(torch.isfinite(got["dr"][1][:, [0, 1, 2, 4, 5, 6, 7]]).all())


# ---- sizes and shapes ------------------------------------------------------

def test_recurrence_in_8_bits_past_4_gib():
    """More than 2^32 elements: the last rows' codes, scales and gradients are
    those of these rows by themselves (tiles begin at the same rows); the norm's
    8-bit output likewise."""
    g = torch.Generator(device="cuda").manual_seed(75)
    R, C, tail = (1 << 22) + 35, 1024, 8192
    cut = (R - tail) // 128 * 128                                    # of a tile
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)        # 8.6 GB
    A, w = -torch.rand(C, device="cuda", generator=g) - 0.01, torch.rand(C, device="cuda", generator=g)
    last = x[cut:].contiguous()
    x[-3:], last[-3:] = -math.inf, -math.inf                         # masked, as r
    _, _, ck, saved = block.glr_forward(x[None], x[None], x[None], A, checkpoint=True, algo="segmented")
    want = block.pack_rows(last)
    for n, p in zip("xri", saved):
        same_rows8(block.Rows8(p.codes[0, cut:], p.scales[0, cut:]), want, n)
    few = [block.Rows8(p.codes[:, cut:].contiguous(), p.scales[:, cut:].contiguous()) for p in saved]
    part = block.glr_backward(*few, A, last[None].nan_to_num(neginf=0.0), ck[cut // 16:].contiguous(), algo="segmented")
    x[-3:] = 0.0
    got = block.glr_backward(*saved, A, x[None], ck, algo="segmented")
    for n in ("dx", "dr", "di"):
        assert torch.equal(got[n][:, cut:], part[n]) and not bool(got[n][:, -3:].any()), n
    del got, saved, ck
    o, p = (block.add_norm_forward(t, None, w, want=("y8",))["y8"] for t in (x[:, :], last.nan_to_num(neginf=0.0)))
    same_rows8(block.Rows8(o.codes[cut:], o.scales[cut:]), p, "y8")


@pytest.mark.parametrize("dtype", list(DT))
def test_every_code_at_every_scale(dtype):
    """Exact in fp32; scale byte 255 is the type's NaN."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8)
    got = block.unpack_rows(block.Rows8(codes.cuda().view(block.CODES), scales.cuda().view(block.SCALES)), DT[dtype]).cpu()
    want = codes.view(block.CODES).double() * torch.exp2(scales[:, :1].double() - 127)
    want[255] = math.nan
    want = want.float().to(DT[dtype])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])


def test_rows_without_leading_dimensions():
    g = gen(76)
    x, res, dy, w = rn(g, 70), rn(g, 70), rn(g, 70), rn(g, 70)
    o, many = block.add_norm_forward(x, res, w, want=("h", "y", "h8")), block.add_norm_forward(x[None], res[None], w, want=("h", "y", "h8"))
    assert torch.equal(o["h"], many["h"][0]) and torch.equal(o["y"], many["y"][0])
    same_rows8(block.pack_rows(o["h"]), o["h8"], "h8")
    assert torch.equal(block.unpack_rows(o["h8"]), block.unpack_rows(many["h8"])[0])
    a, b = block.add_norm_backward(o["h"], dy, None, w), block.add_norm_backward(many["h"], dy[None], None, w)
    assert torch.equal(a["dx"], b["dx"][0]) and torch.equal(a["dweight"], b["dweight"])


def test_mixed_stream_in_place():
    """bf16 rows on an fp32 stream that is updated in place, forwards and backwards."""
    g = gen(77)
    x, dy = rn(g, 9, 136, dtype=torch.bfloat16), rn(g, 9, 136, dtype=torch.bfloat16)
    res, dh, w = rn(g, 9, 136), rn(g, 9, 136), rn(g, 136)
    want = block.add_norm_forward(x, res, w)
    stream = res.clone()
    got = block.add_norm_forward(x, stream, w, out={"h": stream})
    assert torch.equal(stream, want["h"]) and torch.equal(got["y"], want["y"])
    grads = block.add_norm_backward(stream, dy, dh, w)
    into = dh.clone()
    same = block.add_norm_backward(stream, dy, into, w, out={"dresidual": into})
    assert torch.equal(into, grads["dresidual"]) and torch.equal(same["dx"], grads["dx"]) and torch.equal(same["dweight"], grads["dweight"])


@pytest.mark.parametrize("B,T", [(0, 0), (0, 40), (3, 0)])
def test_packed_batches_of_nothing(B, T):
    """No sequences, or sequences without rows: states pass, dA is 0, rows of no
    sequence are left as they were."""
    g = gen(78)
    offsets = torch.zeros(B + 1, dtype=torch.int64).cuda()
    x, r, i, dy = (rn(g, T, 34) for _ in range(4))
    A, h0 = -torch.ones(34).cuda(), rn(g, B, 34)
    rows = {n: torch.full((T, 34), 5.0, device="cuda") for n in ("y", "dx", "dr", "di")}
    _, h, ck, saved = block.glr_forward(x, r, i, A, h0, offsets, out=rows["y"], checkpoint=True)
    assert torch.equal(h, h0) and ck.shape == (block.glr_chunk_count(B, T, True), 34)
    for src in ((x, r, i), saved):
        got = block.glr_backward(*src, A, dy, ck, offsets, h0, out={n: rows[n] for n in ("dx", "dr", "di")})
        assert torch.equal(got["dh0"], h0) and torch.equal(got["dA"], torch.zeros_like(A))
    assert all(bool((t == 5).all()) for t in rows.values())
