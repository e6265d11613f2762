"""The layer operators' 64-bit reference: its gradients against central
differences, and the forms that must agree with each other (CPU)."""
import pytest
import torch

from tests import layer_reference as ref

H = 1e-5


def _rand(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, dtype=torch.float64) * std


def _differences(f, args, wrt, cot):
    """(d <f(args), cot> / d args[wrt] by central differences, their rounding).

    The two sides are sums of magnitude S = sum |o c|, each term off by a few
    roundings (2^-53 relative, 16 counted), and their difference is divided by
    2 H: the quotient is off by up to 16 * 2^-53 S / H."""
    x = args[wrt]
    rounding = 16 * 2.0 ** -53 * float(sum((o * c).abs().sum() for o, c in zip(f(args), cot))) / H
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        side = []
        for sign in (1, -1):
            y = x.clone()
            y.view(-1)[i] += sign * H
            side.append(sum((o * c).sum() for o, c in zip(f({**args, wrt: y}), cot)))
        out.view(-1)[i] = (side[0] - side[1]) / (2 * H)
    return out, rounding


def _agree(got, want, name):
    want, rounding = want
    # the differences' own error is H^2 times a third derivative, O(10) of the value here
    assert torch.allclose(got, want, rtol=1e-7, atol=1e-8 + rounding), (name, (got - want).abs().max())


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("offsets", [None, [1, 1, 3, 3, 7]])
def test_conv_gradients(act, offsets):
    g = torch.Generator().manual_seed(3)
    K, C, B = 4, 2, 2 if offsets is None else 4
    lead = (B, 3) if offsets is None else (8,)
    a = {"x": _rand(g, *lead, C), "weight": _rand(g, C, K), "bias": _rand(g, C), "state0": _rand(g, B, K - 1, C)}
    cot = (_rand(g, *lead, C), _rand(g, B, K - 1, C))
    if offsets is not None:
        cot[0][:1] = cot[0][7:] = 0
    f = lambda v: ref.conv(v["x"], v["weight"], v["bias"], v["state0"], offsets, act)  # noqa: E731
    got = ref.conv_grad(a["x"], a["weight"], cot[0], a["bias"], a["state0"], offsets, act, dstate=cot[1])
    for n, v in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("state0", "dstate0")):
        _agree(got[v], _differences(f, a, n, cot), v)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("offsets", [None, [0, 0, 2, 5]])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients(gate, offsets, softplus):
    g = torch.Generator().manual_seed(4)
    C, N, G, B = 4, 3, 2, 2 if offsets is None else 3
    lead = (B, 4) if offsets is None else (6,)
    a = {"x": _rand(g, *lead, C), "dt": _rand(g, *lead, C), "A": -_rand(g, C, N).abs(), "Bt": _rand(g, *lead, G, N),
         "Ct": _rand(g, *lead, G, N), "skip": _rand(g, C), "z": _rand(g, *lead, C) if gate else None,
         "dt_bias": _rand(g, C), "h0": _rand(g, B, C, N)}
    cot = (_rand(g, *lead, C), _rand(g, B, C, N))
    if offsets is not None:
        cot[0][5:] = 0
    f = lambda v: ref.scan(**v, offsets=offsets, softplus=softplus)[:2]  # noqa: E731
    got = ref.scan_grad(a["x"], a["dt"], a["A"], a["Bt"], a["Ct"], cot[0], a["skip"], a["z"], a["dt_bias"], a["h0"], offsets,
                        softplus, dh_out=cot[1])
    for n in a:
        if a[n] is not None:
            _agree(got["d" + n], _differences(f, a, n, cot), "d" + n)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradients(kind, gate):
    g = torch.Generator().manual_seed(5)
    a = {"x": _rand(g, 3, 5), "weight": _rand(g, 5), "bias": _rand(g, 5), "z": _rand(g, 3, 5) if gate else None}
    cot = (_rand(g, 3, 5),)
    f = lambda v: ref.norm(**v, kind=kind)[:1]  # noqa: E731
    got, bound = ref.norm_grad(a["x"], cot[0], a["weight"], a["bias"], a["z"], kind=kind)
    for n in a:
        if a[n] is not None:
            _agree(got["d" + n], _differences(f, a, n, cot), "d" + n)
            assert bool((got["d" + n].abs() <= bound["d" + n] + 1e-12).all())


def test_absolute_runs_bound_the_values():
    g = torch.Generator().manual_seed(6)
    C, N, G, B, T = 4, 3, 2, 2, 9
    a = dict(x=_rand(g, B, T, C), dt=_rand(g, B, T, C), A=-_rand(g, C, N).abs(), Bt=_rand(g, B, T, G, N),
             Ct=_rand(g, B, T, G, N))
    kw = dict(skip=_rand(g, C), z=_rand(g, B, T, C), dt_bias=_rand(g, C), h0=_rand(g, B, C, N))
    for v, w in zip(ref.scan(**a, **kw)[:2], ref.scan(**a, **kw, absolute=True)[:2]):
        assert bool((v.abs() <= w + 1e-12).all())
    dy = _rand(g, B, T, C)
    v, w = ref.scan_grad(**a, dy=dy, **kw), ref.scan_grad(**a, dy=dy, **kw, absolute=True)
    for n in v:
        assert bool((v[n].abs() <= w[n] + 1e-12).all()), n


def test_segments_continue():
    """Two segments joined by their states equal one sequence."""
    g = torch.Generator().manual_seed(7)
    x, w, b = _rand(g, 1, 9, 3), _rand(g, 3, 4), _rand(g, 3)
    y, st = ref.conv(x, w, b, None, None, "silu")
    y1, s1 = ref.conv(x[:, :2], w, b, None, None, "silu")
    y2, s2 = ref.conv(x[:, 2:], w, b, s1, None, "silu")
    assert torch.allclose(y, torch.cat([y1, y2], 1)) and torch.equal(st, s2)
