"""Plain 64-bit implementations of the layer operators (convolution, scan,
norm) and of their gradients, from the formulas, one sequence and one token at
a time.  CPU, test infrastructure only.

``absolute=True`` runs the same sums over the magnitudes of their terms: the
rounding error of a sum of products is bounded by its magnitude sum times the
number of roundings a term passes through.  ``close`` checks against that
bound plus half a step of the stored type."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24                     # half a step of fp32, relative


def d64(t):
    return None if t is None else t.detach().cpu().to(torch.float64)


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def close(got, want, bound, steps: float, name: str = ""):
    """|got - want| <= half a step of the stored type + steps * 2^-24 * bound."""
    g = d64(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    tol = (half_step(got.dtype) * (1 + 2.0 ** -6) * want.abs() if got.dtype != torch.float32 else 0) + steps * U32 * bound + 1e-36
    bad = ~((g - want).abs() <= tol)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(g[i])!r}, "
                             f"want {float(want[i])!r}, tolerance {float(tol[i])!r}")


def sequences(shape_bt, offsets):
    """Index of each sequence's rows: [b] of a dense batch or a slice."""
    if offsets is None:
        return [b for b in range(shape_bt[0])]
    o = [int(v) for v in offsets]
    return [slice(o[i], max(o[i], o[i + 1])) for i in range(len(o) - 1)]


def silu(v):
    return v * torch.sigmoid(v)


def silu_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


# ---- convolution -----------------------------------------------------------

def conv(x, weight, bias, state0, offsets, act, absolute=False):
    """(y, final state); rows of no sequence are zero in y."""
    x, weight, bias, state0 = d64(x), d64(weight), d64(bias), d64(state0)
    C, K = weight.shape
    if absolute:
        x, weight = x.abs(), weight.abs()
        bias = None if bias is None else bias.abs()
        state0 = None if state0 is None else state0.abs()
    y = torch.zeros_like(x)
    seqs = sequences(x.shape, offsets)
    states = torch.zeros(len(seqs), K - 1, C, dtype=torch.float64)
    for b, at in enumerate(seqs):
        old = torch.zeros(K - 1, C, dtype=torch.float64) if state0 is None else state0[b]
        rows = torch.cat([old, x[at]])
        n = rows.shape[0] - (K - 1)
        p = torch.zeros(n, C, dtype=torch.float64) + (0 if bias is None else bias)
        for k in range(K):
            p = p + rows[k:k + n] * weight[:, k]
        # silu is 1.1-Lipschitz, so its magnitude bound is that of p
        y[at] = p if absolute or act is None else silu(p)
        states[b] = rows[n:]
    return y, states


def conv_grad(x, weight, dy, bias, state0, offsets, act, dstate=None, absolute=False):
    x, weight, dy, bias, state0, dstate = (d64(t) for t in (x, weight, dy, bias, state0, dstate))
    C, K = weight.shape
    pa = conv(x, weight, bias, state0, offsets, None, absolute=True)[0] if absolute else None
    pre = conv(x, weight, bias, state0, offsets, None)[0]
    dp = dy if act is None else dy * silu_slope(pre)
    if absolute:
        # |silu''| <= 0.5: an error of p moves silu' by at most half of it
        dp = dy.abs() * (1.1 + (0 if act is None else pa))
        x, weight = x.abs(), weight.abs()
        state0, dstate = (None if t is None else t.abs() for t in (state0, dstate))
    seqs = sequences(x.shape, offsets)
    g = {"dx": torch.zeros_like(x), "dweight": torch.zeros_like(weight), "dbias": torch.zeros(C, dtype=torch.float64),
         "dstate0": torch.zeros(len(seqs), K - 1, C, dtype=torch.float64)}
    for b, at in enumerate(seqs):
        old = torch.zeros(K - 1, C, dtype=torch.float64) if state0 is None else state0[b]
        rows = torch.cat([old, x[at]])
        n = rows.shape[0] - (K - 1)
        drows = torch.zeros_like(rows)
        for k in range(K):
            g["dweight"][:, k] += (dp[at] * rows[k:k + n]).sum(0)
            drows[k:k + n] += dp[at] * weight[:, k]
        if dstate is not None:
            drows[n:] += dstate[b]
        g["dbias"] += dp[at].sum(0)
        g["dstate0"][b], g["dx"][at] = drows[:K - 1], drows[K - 1:]
    return g


# ---- scan ------------------------------------------------------------------

def _wide(v, C):
    return v.repeat_interleave(C // v.shape[0], 0)       # [G, N] -> [C, N]


def scan(x, dt, A, Bt, Ct, skip=None, z=None, dt_bias=None, h0=None, offsets=None, softplus=True, absolute=False, chunk=32):
    """(y, h after each sequence, recorded states per sequence)."""
    x, dt, A, Bt, Ct, skip, z, dt_bias, h0 = (d64(t) for t in (x, dt, A, Bt, Ct, skip, z, dt_bias, h0))
    ab = torch.abs if absolute else (lambda v: v)
    C, N = A.shape
    seqs = sequences(x.shape, offsets)
    y, last, marks = torch.zeros_like(x), [], []
    for b, at in enumerate(seqs):
        h = torch.zeros(C, N, dtype=torch.float64) if h0 is None else ab(h0[b])
        xs, dts, Bs, Cs = x[at], dt[at], Bt[at], Ct[at]
        out, rec = torch.zeros_like(xs), []
        for t in range(xs.shape[0]):
            if t % chunk == 0:
                rec.append(h)
            raw = dts[t] if dt_bias is None else dts[t] + dt_bias
            d = torch.nn.functional.softplus(raw, threshold=40) if softplus else raw
            h = torch.exp(d[:, None] * A) * h + ab(d * xs[t])[:, None] * ab(_wide(Bs[t], C))
            v = (ab(_wide(Cs[t], C)) * h).sum(1)
            if skip is not None:
                v = v + ab(skip * xs[t])
            out[t] = v if z is None else v * ab(silu(z[at][t]))
        y[at] = out
        last.append(h)
        marks.append(rec)
    return y, torch.stack(last) if last else torch.zeros(0, C, N, dtype=torch.float64), marks


def scan_grad(x, dt, A, Bt, Ct, dy, skip=None, z=None, dt_bias=None, h0=None, offsets=None, softplus=True, dh_out=None,
              absolute=False):
    x, dt, A, Bt, Ct, dy, skip, z, dt_bias, h0, dh_out = (d64(t) for t in (x, dt, A, Bt, Ct, dy, skip, z, dt_bias, h0, dh_out))
    ab = torch.abs if absolute else (lambda v: v)
    C, N = A.shape
    G = Bt.shape[-2]
    seqs = sequences(x.shape, offsets)
    g = {"dx": torch.zeros_like(x), "ddt": torch.zeros_like(x), "dBt": torch.zeros_like(Bt), "dCt": torch.zeros_like(Ct),
         "dz": torch.zeros_like(x), "dA": torch.zeros_like(A), "dskip": torch.zeros(C, dtype=torch.float64),
         "ddt_bias": torch.zeros(C, dtype=torch.float64), "dh0": torch.zeros(len(seqs), C, N, dtype=torch.float64)}
    sk = torch.zeros(C, dtype=torch.float64) if skip is None else ab(skip)
    for b, at in enumerate(seqs):
        xs, dts, Bs, Cs, dys = x[at], dt[at], Bt[at], Ct[at], dy[at]
        n = xs.shape[0]
        raw = dts if dt_bias is None else dts + dt_bias
        d = torch.nn.functional.softplus(raw, threshold=40) if softplus else raw
        slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
        a = torch.exp(d[:, :, None] * A)
        hs = [torch.zeros(C, N, dtype=torch.float64) if h0 is None else ab(h0[b])]
        for t in range(n):
            hs.append(a[t] * hs[-1] + ab(d[t] * xs[t])[:, None] * ab(_wide(Bs[t], C)))
        lam = torch.zeros(C, N, dtype=torch.float64) if dh_out is None else ab(dh_out[b])
        out = {m: torch.zeros_like(g[m][at]) for m in ("dx", "ddt", "dBt", "dCt", "dz")}
        for t in range(n - 1, -1, -1):
            xt, dt_, Bn, Cn = ab(xs[t]), ab(d[t]), ab(_wide(Bs[t], C)), ab(_wide(Cs[t], C))
            dv = ab(dys[t])
            if z is not None:
                zt = z[at][t]
                v = (Cn * hs[t + 1]).sum(1) + sk * xt
                # |silu''| <= 0.5 is part of the slope's magnitude
                out["dz"][t] = dv * v * (ab(silu_slope(zt)) if not absolute else 1.1)
                dv = dv * ab(silu(zt))
            lam = lam + dv[:, None] * Cn
            out["dCt"][t] = (dv[:, None] * hs[t + 1]).view(G, C // G, N).sum(1)
            out["dBt"][t] = (lam * (dt_ * xt)[:, None]).view(G, C // G, N).sum(1)
            du = (lam * Bn).sum(1)
            q = lam * a[t] * hs[t]
            dd = (du * xt + (q * ab(A)).sum(1)) * slope[t]
            out["dx"][t] = du * dt_ + sk * dv
            out["ddt"][t] = dd
            g["dA"] += q * dt_[:, None]
            g["dskip"] += dv * xt
            g["ddt_bias"] += dd
            lam = lam * a[t]
        for m, v in out.items():
            g[m][at] = v
        g["dh0"][b] = lam
    return g


# ---- norm ------------------------------------------------------------------

def norm(x, weight=None, bias=None, z=None, eps=1e-5, kind="layer"):
    """(y, bound of y's terms)."""
    x, weight, bias, z = d64(x), d64(weight), d64(bias), d64(z)
    C = x.shape[-1]
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight
    b = torch.zeros(C, dtype=torch.float64) if bias is None else bias
    m = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    r = ((x - m).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (x - m) * r
    xa = (x.abs() + (x.abs().mean(-1, keepdim=True) if kind == "layer" else 0)) * r
    y, bound = xh * w + b, xa * w.abs() * (2 + xa) + b.abs()
    if z is not None:
        y, bound = y * silu(z), bound * silu(z).abs()
    return y, bound


def norm_grad(x, dy, weight=None, bias=None, z=None, eps=1e-5, kind="layer"):
    """(gradients, bounds of their terms)."""
    x, dy, weight, bias, z = d64(x), d64(dy), d64(weight), d64(bias), d64(z)
    C = x.shape[-1]
    w = torch.ones(C, dtype=torch.float64) if weight is None else weight
    b = torch.zeros(C, dtype=torch.float64) if bias is None else bias
    layer = kind == "layer"
    m = x.mean(-1, keepdim=True) if layer else torch.zeros_like(x[..., :1])
    r = ((x - m).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (x - m) * r
    xa = (x.abs() + (x.abs().mean(-1, keepdim=True) if layer else 0)) * r
    amp = 2 + xa
    g, bd = {}, {}
    dn = dy
    if z is not None:
        n = xh * w + b
        g["dz"], bd["dz"] = dy * n * silu_slope(z), dy.abs() * (xa * w.abs() * amp + b.abs()) * 1.1
        dn = dy * silu(z)
    v = dn * w
    g["dx"] = r * (v - (v.mean(-1, keepdim=True) if layer else 0) - xh * (v * xh).mean(-1, keepdim=True))
    va = v.abs()
    bd["dx"] = r * (va + va.mean(-1, keepdim=True) + xa * (va * xa * amp).mean(-1, keepdim=True)) * amp
    flat = lambda t: t.reshape(-1, C).sum(0)  # noqa: E731
    g["dweight"], bd["dweight"] = flat(dn * xh), flat(dn.abs() * xa * amp)
    g["dbias"], bd["dbias"] = flat(dn), flat(dn.abs())
    return g, bd
