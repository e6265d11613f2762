"""Plain 64-bit implementations of the block operators (rows in 8 bits, norm
with the residual's addition, gated linear recurrence) and of their gradients,
from the formulas, one sequence and one token at a time.  CPU, test
infrastructure only; tests/layer_reference.py holds the tolerance's rule.

The recurrence's bounds: a decay that is off by k roundings (k 2^-24 of its
value) changes the state by that share of what it multiplies, in every token.
With H the state of the magnitudes, the error of h is then at most k 2^-24 M,
    M_t = a_t (M_{t-1} + H_{t-1}) + |b_t|,
and the gradient's, walking backwards, likewise."""
from __future__ import annotations

import math

import torch

from tests.layer_reference import d64, sequences

BLOCK = 32
CHUNK = 16


# ---- rows in 8 bits --------------------------------------------------------

def e4m3(t: float) -> float:
    """The nearest e4m3 number, ties to even, of a value of at most 448."""
    if t == 0 or math.isnan(t):
        return t
    step = math.ldexp(1.0, max(math.frexp(t)[1] - 1, -6) - 3)
    n = t / step                       # exact: a power of two
    f = math.floor(n)
    up = n - f > 0.5 or (n - f == 0.5 and f % 2 == 1)
    return (f + up) * step


def exponent(block) -> int:
    """The smallest e >= -127 with max |v| <= 448 2^e over the finite values; 120 without any."""
    some = [abs(v) for v in block if math.isfinite(v)]
    if not some:
        return 120
    e = -127
    while max(some) > math.ldexp(448.0, e):
        e += 1
    return e


def pack(x):
    """(codes, exponents, values) of [R, C] rows."""
    rows = d64(x).reshape(-1, x.shape[-1])
    codes, values = torch.empty_like(rows), torch.empty_like(rows)
    nb = -(-rows.shape[1] // BLOCK)
    exps = torch.empty(rows.shape[0], nb, dtype=torch.int64)
    for r in range(rows.shape[0]):
        for b in range(nb):
            block = [float(v) for v in rows[r, b * BLOCK:(b + 1) * BLOCK]]
            e = exponent(block)
            some = any(math.isfinite(v) for v in block)
            exps[r, b] = e
            for j, v in enumerate(block):
                if math.isinf(v):
                    c = math.copysign(448.0, v) if not some else math.nan
                else:
                    c = e4m3(math.ldexp(v, -e))
                codes[r, b * BLOCK + j] = c
                value = c * 2.0 ** e
                values[r, b * BLOCK + j] = math.copysign(math.inf, value) if abs(value) >= 2.0 ** 128 else value
    lead = x.shape[:-1]
    return codes.reshape(x.shape), exps.reshape(*lead, nb), values.reshape(x.shape)


# ---- norm with the residual's addition -------------------------------------

def add(x, residual):
    """The stream as it is stored, in 64 bits."""
    if residual is None:
        return d64(x)
    return (d64(x) + d64(residual)).to(residual.dtype).to(torch.float64)


def held(eps: float) -> float:
    """eps as the C ABI holds it, in fp32: 1e-3 is 4.7e-11 larger there, which moves n by up to
    4.7e-11 / (2 (var + eps)) of its value, more than the 64-bit norm is held to."""
    return float(torch.tensor(eps, dtype=torch.float32))


def norm(h, weight, bias, eps, kind):
    C, eps = h.shape[-1], held(eps)
    w = torch.ones(C, dtype=torch.float64) if weight is None else d64(weight)
    b = torch.zeros(C, dtype=torch.float64) if bias is None else d64(bias)
    m = h.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(h[..., :1])
    r = ((h - m).square().mean(-1, keepdim=True) + eps) ** -0.5
    return (h - m) * r * w + b


def norm_grad(h, dy, dh, weight, eps, kind):
    """({dresidual, dweight, dbias}, bounds of their terms)."""
    from tests import layer_reference
    w = None if weight is None else d64(weight)
    g, bd = layer_reference.norm_grad(h, d64(dy), w, None, None, held(eps), kind)
    more = torch.zeros_like(h) if dh is None else d64(dh)
    return ({"dresidual": g["dx"] + more, "dweight": g["dweight"], "dbias": g["dbias"]},
            {"dresidual": bd["dx"] + more.abs(), "dweight": bd["dweight"], "dbias": bd["dbias"]})


# ---- gated linear recurrence -----------------------------------------------

def terms(x, r, i, A):
    """(s(r), s(i), a, q, b) of [t, c] rows."""
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    u = torch.where(sr == 0, torch.zeros_like(r), A * sr)
    a, q = torch.exp(u), torch.sqrt(-torch.expm1(2 * u))
    return sr, si, a, q, torch.where(q == 0, torch.zeros_like(x), q * si * x)


def glr(x, r, i, A, h0=None, offsets=None):
    """(y, bound of y, h after each sequence, its bound, states before every
    16th token per sequence); rows of no sequence are zero in y."""
    x, r, i, A, h0 = (d64(t) for t in (x, r, i, A, h0))
    C = A.shape[0]
    seqs = sequences(x.shape, offsets)
    y, bound, last, lastb, marks = torch.zeros_like(x), torch.zeros_like(x), [], [], []
    for s, at in enumerate(seqs):
        h = torch.zeros(C, dtype=torch.float64) if h0 is None else h0[s]
        H, M, rec = h.abs(), h.abs(), []
        _, _, a, _, b = terms(x[at], r[at], i[at], A)
        out, ob = torch.zeros_like(b), torch.zeros_like(b)
        for t in range(b.shape[0]):
            if t % CHUNK == 0:
                rec.append((h, M))
            M, H = a[t] * (M + H) + b[t].abs(), a[t] * H + b[t].abs()
            h = a[t] * h + b[t]
            out[t], ob[t] = h, M
        y[at], bound[at] = out, ob
        last.append(h), lastb.append(M), marks.append(rec)
    empty = torch.zeros(0, C, dtype=torch.float64)
    return y, bound, torch.stack(last) if last else empty, torch.stack(lastb) if lastb else empty, marks


def glr_grad(x, r, i, A, dy, h0=None, offsets=None, dh_out=None, starts=None):
    """Gradients and bounds of their terms.  ``starts``: per sequence, the
    states before every 16th token to form the others from (the gradients from
    rows in 8 bits); by default they follow from h0."""
    x, r, i, A, dy, h0, dh_out = (d64(t) for t in (x, r, i, A, dy, h0, dh_out))
    C = A.shape[0]
    seqs = sequences(x.shape, offsets)
    g = {n: torch.zeros_like(x) for n in ("dx", "dr", "di")}
    bd = {n: torch.zeros_like(x) for n in g}
    for d in (g, bd):
        d["dA"], d["dh0"] = torch.zeros(C, dtype=torch.float64), torch.zeros(len(seqs), C, dtype=torch.float64)
    for s, at in enumerate(seqs):
        sr, si, a, q, b = terms(x[at], r[at], i[at], A)
        n = b.shape[0]
        h = torch.zeros(C, dtype=torch.float64) if h0 is None else h0[s]
        H, M = h.abs(), h.abs()
        hp, Mp = torch.zeros_like(b), torch.zeros_like(b)
        for t in range(n):
            if starts is not None and t % CHUNK == 0:
                h, M = starts[s][t // CHUNK]
                H = h.abs()
            hp[t], Mp[t] = h, M + H
            M, H, h = a[t] * (M + H) + b[t].abs(), a[t] * H + b[t].abs(), a[t] * h + b[t]
        lam = torch.zeros(C, dtype=torch.float64) if dh_out is None else dh_out[s]
        G, Mg = lam.abs(), lam.abs()
        shut = q == 0
        xs, o = x[at].masked_fill(shut, 0.0), si.masked_fill(shut, 0.0)
        over = torch.where(shut, torch.zeros_like(q), a * a / q)
        rows = {m: torch.zeros_like(b) for m in ("dx", "dr", "di")}
        rb = {m: torch.zeros_like(b) for m in rows}
        for t in range(n - 1, -1, -1):
            gt, Gt, Mt = dy[at][t] + lam, dy[at][t].abs() + G, dy[at][t].abs() + Mg + G
            du = gt * (a[t] * hp[t] - o[t] * xs[t] * over[t])
            dub = Mt * (a[t] * Mp[t] + (o[t] * xs[t] * over[t]).abs())
            rows["dx"][t], rb["dx"][t] = gt * q[t] * o[t], Mt * q[t] * o[t]
            rows["di"][t], rb["di"][t] = gt * q[t] * o[t] * xs[t] * (1 - o[t]), Mt * q[t] * o[t] * xs[t].abs()
            slope = A * sr[t] * (1 - sr[t])
            rows["dr"][t], rb["dr"][t] = du * slope, dub * A.abs() * sr[t]
            g["dA"] += du * sr[t]
            bd["dA"] += dub * sr[t]
            lam, G, Mg = a[t] * gt, a[t] * Gt, a[t] * Mt
        g["dh0"][s], bd["dh0"][s] = lam, Mg + G
        for m in rows:
            g[m][at], bd[m][at] = rows[m], rb[m]
    return g, bd
