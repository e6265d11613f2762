"""The 64-bit implementations the block operators are held to, checked by
other means (no GPU needed): automatic differentiation, differences, torch's
own 8-bit type, and cases with a closed form."""
import math

import pytest
import torch

from tests import block_reference as ref

F64 = torch.float64


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, dtype=F64) * std


def test_codes_are_the_nearest_of_all():
    """Every code's value and every middle between two neighbours."""
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    for k in range(126):
        a, b = float(grid[k]), float(grid[k + 1])
        assert ref.e4m3(a) == a and ref.e4m3(-a) == -a
        mid = (a + b) / 2
        assert ref.e4m3(mid) == (a if k % 2 == 0 else b)
        assert ref.e4m3(mid - 1e-9 * b) == a and ref.e4m3(mid + 1e-9 * b) == b and ref.e4m3(-mid - 1e-9 * b) == -b
    t = torch.randn(4000, generator=gen(1)) * 20
    assert [ref.e4m3(float(v)) for v in t] == t.to(torch.float8_e4m3fn).double().tolist()


@pytest.mark.parametrize("most,e", [(448.0, 0), (448.5, 1), (447.0, 0), (224.0, -1), (0.0, -127), (1.75, -8), (1.76, -7),
                                    (3.3e38, 120), (1e-45, -127), (2.0 ** -118, -126), (1.75 * 2.0 ** -118, -126),
                                    (1.75 * 2.0 ** -119, -127)])
def test_exponents(most, e):
    assert ref.exponent([0.0, -most, most / 2, math.nan, math.inf]) == e


def test_blocks_without_finite_values():
    inf, nan = math.inf, math.nan
    codes, exps, values = ref.pack(torch.tensor([[-inf] * 3 + [nan], [-inf, 1.0, inf, nan]]))
    assert exps.tolist() == [[120], [-8]]
    assert values[0, :3].tolist() == [-inf] * 3 and math.isnan(values[0, 3]) and codes[0, 0] == -448
    assert torch.isnan(values[1, [0, 2, 3]]).all() and values[1, 1] == 1.0
    # the lowest numbers of both types read as -inf
    for t in (torch.bfloat16, torch.float32):
        assert ref.pack(torch.full((1, 5), torch.finfo(t).min, dtype=t))[2].tolist() == [[-inf] * 5]


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_gradients(kind):
    g = gen(2)
    x, res, w, b, dy, dh = rn(g, 5, 7), rn(g, 5, 7), rn(g, 7), rn(g, 7), rn(g, 5, 7), rn(g, 5, 7)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    h = leaves[0] + res
    n = (h - h.mean(1, keepdim=True) if kind == "layer" else h)
    n = n * (n.square().mean(1, keepdim=True) + ref.held(1e-3)) ** -0.5 * leaves[1] + leaves[2]
    assert torch.allclose(ref.norm(h.detach(), w, b, 1e-3, kind), n.detach(), rtol=1e-13)
    want = torch.autograd.grad((n * dy).sum() + (h * dh).sum(), leaves)
    got, bound = ref.norm_grad(h.detach(), dy, dh, w, 1e-3, kind)
    for n_, v in zip(("dresidual", "dweight", "dbias"), want):
        assert torch.allclose(got[n_], v, rtol=1e-12, atol=1e-12), n_
        assert bool((bound[n_] * (1 + 1e-12) >= v.abs()).all()), n_


OFFSETS = torch.tensor([1, 1, 6, 7, 26, 26])


def case(seed, packed):
    g = gen(seed)
    lead, B = ((28,), 5) if packed else ((2, 19), 2)
    A = -torch.rand(3, generator=g, dtype=F64) - 0.05
    return (rn(g, *lead, 3), rn(g, *lead, 3), rn(g, *lead, 3), A), rn(g, *lead, 3), rn(g, B, 3), rn(g, B, 3), OFFSETS if packed else None


def loss_of(rows, A, h0, offsets, dy, dh):
    y, _, last, _, _ = ref.glr(*rows, A, h0, offsets)
    return (y * dy).sum() + (last * dh).sum()


@pytest.mark.parametrize("packed", [False, True])
def test_glr_gradients_by_differences(packed):
    (x, r, i, A), dy, h0, dh, offsets = case(3, packed)
    g, bound = ref.glr_grad(x, r, i, A, dy, h0, offsets, dh)
    args = {"dx": x, "dr": r, "di": i, "dA": A, "dh0": h0}
    pick = gen(4)
    for n, t in args.items():
        assert bool((bound[n] * (1 + 1e-9) >= g[n].abs()).all()), n
        for _ in range(12):
            at = tuple(int(torch.randint(0, s, (1,), generator=pick)) for s in t.shape)
            d = []
            for sign in (1, -1):
                moved = {k: v.clone() for k, v in args.items()}
                moved[n][at] += sign * 1e-6
                d.append(loss_of((moved["dx"], moved["dr"], moved["di"]), moved["dA"], moved["dh0"], offsets, dy, dh))
            assert float((d[0] - d[1]) / 2e-6) == pytest.approx(float(g[n][at]), rel=1e-6, abs=1e-8), (n, at)


def test_glr_gradients_by_autograd():
    """The recurrence unrolled under automatic differentiation."""
    (x, r, i, A), dy, h0, dh, _ = case(5, False)
    leaves = [t.clone().requires_grad_() for t in (x, r, i, A, h0)]
    u = leaves[3] * torch.sigmoid(leaves[1])
    a, b = torch.exp(u), torch.sqrt(-torch.expm1(2 * u)) * torch.sigmoid(leaves[2]) * leaves[0]
    h, loss = leaves[4], 0.0
    for t in range(x.shape[1]):
        h = a[:, t] * h + b[:, t]
        loss = loss + (h * dy[:, t]).sum()
    want = torch.autograd.grad(loss + (h * dh).sum(), leaves)
    got, _ = ref.glr_grad(x, r, i, A, dy, h0, None, dh)
    for n, v in zip(("dx", "dr", "di", "dA", "dh0"), want):
        assert torch.allclose(got[n], v, rtol=1e-11, atol=1e-13), n


def test_glr_masked_tokens():
    """A masked token is as if it were not there, whatever it holds."""
    (x, r, i, A), dy, h0, dh, _ = case(6, False)
    keep = torch.ones(19, dtype=torch.bool)
    keep[[0, 4, 5, 18]] = False
    mx, mr, mi = x.clone(), r.clone(), i.clone()
    mr[:, ~keep] = -math.inf
    mx[:, 4], mi[:, 5], mx[:, 18] = math.nan, math.nan, math.inf
    mdy = dy.clone()
    mdy[:, ~keep] = 0
    y, _, last, _, _ = ref.glr(mx, mr, mi, A, h0)
    y2, _, last2, _, _ = ref.glr(x[:, keep], r[:, keep], i[:, keep], A, h0)
    assert torch.equal(y[:, keep], y2) and torch.equal(last, last2)
    g, _ = ref.glr_grad(mx, mr, mi, A, mdy, h0, None, dh)
    g2, _ = ref.glr_grad(x[:, keep], r[:, keep], i[:, keep], A, dy[:, keep], h0, None, dh)
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][:, keep], g2[n]) and not bool(g[n][:, ~keep].any()), n
    assert torch.allclose(g["dA"], g2["dA"]) and torch.equal(g["dh0"], g2["dh0"])


def test_glr_constant_input():
    """r = +inf: a = e^A in every token, a geometric series."""
    A = torch.tensor([-0.3], dtype=F64)
    x, r, i = torch.full((1, 9, 1), 2.0, dtype=F64), torch.full((1, 9, 1), math.inf, dtype=F64), torch.full((1, 9, 1), math.inf, dtype=F64)
    a = math.exp(-0.3)
    y = ref.glr(x, r, i, A)[0]
    for t in range(9):
        assert float(y[0, t, 0]) == pytest.approx(2 * math.sqrt(1 - a * a) * (1 - a ** (t + 1)) / (1 - a), rel=1e-13)
