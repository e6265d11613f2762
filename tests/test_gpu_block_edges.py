"""GPU tests of the block operators at calls their documentation allows and
tests/test_gpu_block.py does not make, against the same 64-bit implementation
and with its tolerances."""
import math

import pytest
import torch

from gated_delta_rule_86_amd import block
from tests import block_reference as ref
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
