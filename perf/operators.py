"""Cases of the operators around the recurrence: the short causal
convolution, the selective state space scan and the normalisation of a
sequence-mixing layer, each over whole prompts, packed batches, single tokens
and (for training) backwards.

`run` computes a case either through the package's entry points (`own` true)
or in plain torch operations in 32 bits; `exact` gives the same outputs in 64
bits from the operators' definitions.

Definitions (t runs over the tokens of one sequence, c over channels):

  convolution   p[t,c] = bias[c] + sum_k weight[c,k] x[t-(K-1)+k, c], where the
                rows before the sequence come from its state [K-1, c] (zero
                without one);  y = silu(p).  The final state is the last K-1
                rows of (state, x).
  scan          d = softplus(dt + dt_bias);  h_t = exp(d A) h_{t-1} + d x B_t
                (h, A: [channel, state]; B_t, C_t: [group, state], shared by
                the channels of a group);  y = (C_t . h_t + skip x) silu(z)
  normalisation n = (x - m) / sqrt(mean((x - m)^2) + eps) weight + bias, m the
                row's mean ("layer") or 0 ("rms");  y = n, or n silu(z)
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


def listed():
    return [
        # The convolution before the mixer at the benchmark's training shape (8 x 4096 tokens, 16 heads of
        # 128): x is one half of an input projection's rows, as a layer hands it on.
        {"name": "conv_prompt", "op": "conv", "B": 8, "T": 4096, "C": 2048, "K": 4, "dtype": "bf16", "packed": False,
         "init": False},
        # A decode step of the benchmark's 256 sequences through the convolution.
        {"name": "conv_step", "op": "conv_step", "B": 256, "C": 2048, "K": 4, "dtype": "bf16"},
        # The convolution's gradients at the training shape.
        {"name": "conv_backward", "op": "conv_backward", "B": 8, "T": 4096, "C": 2048, "K": 4, "dtype": "bf16",
         "packed": False, "init": False},
        # A ragged packed batch in fp32 that continues earlier segments: odd channel count, three taps.
        {"name": "conv_backward_packed", "op": "conv_backward", "B": 13, "T": 10007, "C": 1003, "K": 3, "dtype": "f32",
         "packed": True, "init": True},
        # The scan over the training shape's prompts, gated, state 16.
        {"name": "scan_prompt", "op": "scan", "B": 8, "T": 4096, "C": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "packed": False, "init": False, "gate": True},
        # One long prompt that continues a state: few rows, many tokens.
        {"name": "scan_long", "op": "scan", "B": 1, "T": 32768, "C": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "packed": False, "init": True, "gate": True},
        # Serving a ragged packed batch in fp32: odd sizes, two groups, a state that is no power of two.
        {"name": "scan_packed", "op": "scan", "B": 9, "T": 5003, "C": 1002, "N": 12, "G": 2, "dtype": "f32",
         "packed": True, "init": True, "gate": False},
        # One training step of the scan: forward, then every gradient.
        {"name": "scan_train", "op": "scan_train", "B": 4, "T": 2048, "C": 2048, "N": 16, "G": 1, "dtype": "bf16",
         "packed": False, "gate": True},
        # One token of one sequence: the smallest call, all latency.
        {"name": "scan_step_one", "op": "scan_step", "B": 1, "C": 2048, "N": 16, "G": 1, "dtype": "bf16", "gate": True},
        # A decode step of 256 sequences.
        {"name": "scan_step", "op": "scan_step", "B": 256, "C": 2048, "N": 16, "G": 1, "dtype": "bf16", "gate": True},
        # The gated per-head norm of the mixer's output at the training shape (8 x 4096 x 16 rows of 128).
        {"name": "norm_heads", "op": "norm", "R": 524288, "C": 128, "dtype": "bf16", "kind": "rms", "gate": True},
        # The gradients of a block's layer norm at the training shape.
        {"name": "norm_backward", "op": "norm_backward", "R": 32768, "C": 2048, "dtype": "bf16", "kind": "layer",
         "gate": False},
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "conv_backward", "scan", "scan_train", "scan_step", "norm", "norm_backward"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    half = 2 if c["dtype"] == "f32" else 1
    if op in ("norm", "norm_backward"):
        c["kind"] = rng.choice(["layer", "rms"])
        c["gate"] = rng.random() < 0.4
        c["C"] = _logint(rng, 33, 8192)
        c["R"] = _logint(rng, 1, max(1, min(524288, (1 << 25) // (half * c["C"]))))
        return c
    c["C"] = _logint(rng, 64, 4096)
    if op.startswith("conv"):
        c["K"] = rng.choice([2, 3, 4, 4])
    else:
        c["G"] = rng.choice([1, 1, 2])
        c["C"] -= c["C"] % c["G"]
        c["N"] = rng.choice([4, 8, 11, 16, 16, 16, 32])
        c["gate"] = rng.random() < 0.6
    if op.endswith("_step"):
        c["B"] = _logint(rng, 1, 256)
        return c
    c["packed"] = rng.random() < 0.4
    if op != "scan_train":
        c["init"] = rng.random() < 0.5
    most = (1 << 26) // half if op.startswith("conv") else (1 << 22) // half if op == "scan_train" else (1 << 24) // half
    most = max(1, most // c["C"])
    c["B"] = rng.randint(2, 16) if c["packed"] else _logint(rng, 1, 16)
    if c["packed"]:
        c["T"] = _logint(rng, min(64, most), min(16384, most))
    else:
        c["T"] = _logint(rng, 1, max(1, min(8192, most // c["B"])))
    return c


# ---------------------------------------------------------------- inputs

def _offsets(B, T, seed):
    """B + 1 ascending offsets over T rows; about one sequence in eight is empty."""
    r = random.Random(seed * 7919 + 13)
    cuts = sorted(r.randint(0, T) for _ in range(B - 1))
    offs = [0] + cuts + [T]
    for i in range(1, B):
        if r.random() < 0.125:
            offs[i] = offs[i - 1]
    return offs


def prepare(case, seed):
    dev, dt = _dev(), DTYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def rn(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    def ru(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device=dev) * (hi - lo) + lo

    op, C = case["op"], case["C"]
    s = {"case": case, "op": op}
    if op in ("norm", "norm_backward"):
        R = case["R"]
        s["x"] = rn(R, C) * 1.5 + 0.25
        s["weight"] = 1.0 + 0.1 * rn(C, dtype=torch.float32)
        s["bias"] = 0.1 * rn(C, dtype=torch.float32) if case["kind"] == "layer" else None
        s["z"] = rn(R, C) if case["gate"] else None
        s["dy"] = rn(R, C) if op == "norm_backward" else None
        return s
    B = case["B"]
    if op.startswith("conv"):
        K = case["K"]
        s["weight"] = ru(C, K, lo=-1.0, hi=1.0) / math.sqrt(K)
        s["bias"] = ru(C, lo=-0.5, hi=0.5)
    else:
        N, G = case["N"], case["G"]
        s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32).repeat(C, 1) * ru(C, N, lo=0.7, hi=1.3)
        s["skip"] = 1.0 + 0.1 * rn(C, dtype=torch.float32)
        # softplus(dt_bias) spread over 0.001 .. 0.1 on a logarithmic scale
        step = torch.exp(ru(C, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    if op == "conv_step":
        s["state"], s["x"] = rn(B, K - 1, C), rn(B, 2 * C)[:, :C]
        return s
    if op == "scan_step":
        proj = rn(B, 2 * G * N)
        s["state"] = rn(B, C, N, std=0.3, dtype=torch.float32)
        s["x"], s["dt"] = rn(B, C), rn(B, C)
        s["Bt"], s["Ct"] = proj[:, :G * N].unflatten(1, (G, N)), proj[:, G * N:].unflatten(1, (G, N))
        s["z"] = rn(B, 2 * C)[:, C:] if case["gate"] else None
        return s
    T, packed = case["T"], case["packed"]
    lead = (T,) if packed else (B, T)
    s["offs"] = _offsets(B, T, int(seed)) if packed else None
    s["offsets"] = torch.tensor(s["offs"], dtype=torch.int64, device=dev) if packed else None
    if op.startswith("conv"):
        s["x"] = rn(*lead, 2 * C)[..., :C]
        s["state0"] = rn(B, K - 1, C) if case["init"] else None
        if op == "conv_backward":
            s["dy"] = rn(*lead, C)
        return s
    proj = rn(*lead, 2 * G * N)
    x = rn(*lead, C, dtype=torch.float32)
    s["x"] = (x * torch.sigmoid(x)).to(dt)
    s["dt"] = rn(*lead, C)
    s["Bt"], s["Ct"] = proj[..., :G * N].unflatten(-1, (G, N)), proj[..., G * N:].unflatten(-1, (G, N))
    s["z"] = rn(*lead, 2 * C)[..., C:] if case["gate"] else None
    s["h0"] = rn(B, C, N, std=0.3, dtype=torch.float32) if case.get("init") else None
    if op == "scan_train":
        s["dy"] = rn(*lead, C)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _OWN[state["op"]](state) if own else _PLAIN[state["op"]](state)


def _own_conv(s):
    from gated_delta_rule_86_amd import layer
    return layer.conv_forward(s["x"], s["weight"], s["bias"], state0=s["state0"], offsets=s["offsets"])


def _own_conv_step(s):
    from gated_delta_rule_86_amd import layer
    return layer.conv_step(s["state"], s["x"], s["weight"], s["bias"]), s["state"]


def _own_conv_backward(s):
    from gated_delta_rule_86_amd import layer
    return layer.conv_backward(s["x"], s["weight"], s["dy"], s["bias"], state0=s["state0"], offsets=s["offsets"])


def _own_scan(s):
    from gated_delta_rule_86_amd import layer
    return layer.scan_forward(s["x"], s["dt"], s["A"], s["Bt"], s["Ct"], skip=s["skip"], z=s["z"],
                              dt_bias=s["dt_bias"], h0=s["h0"], offsets=s["offsets"])


def _own_scan_step(s):
    from gated_delta_rule_86_amd import layer
    y = layer.scan_step(s["state"], s["x"], s["dt"], s["A"], s["Bt"], s["Ct"], skip=s["skip"], z=s["z"],
                        dt_bias=s["dt_bias"])
    return y, s["state"]


def _own_scan_train(s):
    from gated_delta_rule_86_amd import layer
    a = (s["x"], s["dt"], s["A"], s["Bt"], s["Ct"])
    kw = dict(skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], offsets=s["offsets"])
    y, _, chunks = layer.scan_forward(*a, final_state=False, chunk_states=True, **kw)
    grads = layer.scan_backward(*a, dy=s["dy"], h_chunks=chunks, want_dh0=False, **kw)
    return y, grads


def _own_norm(s):
    from gated_delta_rule_86_amd import layer
    return layer.norm_forward(s["x"], s["weight"], s["bias"], z=s["z"], eps=EPS, kind=s["case"]["kind"])


def _own_norm_backward(s):
    from gated_delta_rule_86_amd import layer
    return layer.norm_backward(s["x"], s["dy"], s["weight"], s["bias"], z=s["z"], eps=EPS, kind=s["case"]["kind"])


_OWN = {"conv": _own_conv, "conv_step": _own_conv_step, "conv_backward": _own_conv_backward, "scan": _own_scan,
        "scan_step": _own_scan_step, "scan_train": _own_scan_train, "norm": _own_norm,
        "norm_backward": _own_norm_backward}


# ---------------------------------------------------------------- plain forms (32 bits)

def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _starts(s, rows):
    """Packed rows' sequence and position, from the offsets (a dense batch is rows of equal sequences)."""
    row = torch.arange(rows, device=s["x"].device)
    seq = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True)
    return seq, row - s["offsets"][seq]


def _plain_taps(s):
    """The K shifted inputs of the convolution, in 32 bits, and where each comes from."""
    x, K = s["x"].float(), s["weight"].shape[1]
    if s["offsets"] is None:
        B, T, C = x.shape
        st = torch.zeros(B, K - 1, C, device=x.device) if s["state0"] is None else s["state0"].float()
        pad = torch.cat([st, x], 1)
        return [pad[:, k:k + T] for k in range(K)]
    seq, pos = _starts(s, x.shape[0])
    row = torch.arange(x.shape[0], device=x.device)
    taps = []
    for k in range(K):
        back = K - 1 - k
        v = torch.where((pos >= back)[:, None], x[(row - back).clamp(min=0)], torch.zeros_like(x))
        if s["state0"] is not None:
            old = s["state0"].float()[seq, (pos + k).clamp(max=K - 2)]
            v = torch.where((pos < back)[:, None], old, v)
        taps.append(v)
    return taps


def _plain_final(s):
    """The last K - 1 rows of (state, sequence)."""
    x, K = s["x"], s["weight"].shape[1]
    B, C = s["case"]["B"], x.shape[-1]
    st = torch.zeros(B, K - 1, C, device=x.device, dtype=x.dtype) if s["state0"] is None else s["state0"]
    if s["offsets"] is None:
        return torch.cat([st, x], 1)[:, -(K - 1):].contiguous()
    rows = []
    for b in range(B):
        rows.append(torch.cat([st[b], x[s["offs"][b]:s["offs"][b + 1]]])[-(K - 1):])
    return torch.stack(rows)


def _plain_conv(s):
    w = s["weight"]
    p = s["bias"] + sum(t * w[:, k] for k, t in enumerate(_plain_taps(s)))
    return (p * torch.sigmoid(p)).to(s["x"].dtype), _plain_final(s)


def _plain_conv_step(s):
    st, x, w = s["state"], s["x"], s["weight"]
    full = torch.cat([st, x[:, None]], 1)
    p = s["bias"] + (full.float() * w.t()).sum(1)
    st.copy_(full[:, 1:])
    return (p * torch.sigmoid(p)).to(x.dtype), st


def _plain_conv_backward(s):
    x, w, K = s["x"], s["weight"], s["weight"].shape[1]
    taps = _plain_taps(s)
    p = s["bias"] + sum(t * w[:, k] for k, t in enumerate(taps))
    sg = torch.sigmoid(p)
    dp = s["dy"].float() * sg * (1 + p * (1 - sg))
    C = w.shape[0]
    dw = torch.stack([(dp * t).reshape(-1, C).sum(0) for t in taps], 1)
    db = dp.reshape(-1, C).sum(0)
    B, dst = s["case"]["B"], None
    if s["offsets"] is None:
        T = x.shape[1]
        dpad = torch.zeros(B, T + K - 1, C, device=x.device)
        for k in range(K):
            dpad[:, k:k + T] += dp * w[:, k]
        dx = dpad[:, K - 1:]
        dst = dpad[:, :K - 1]
    else:
        T = x.shape[0]
        seq, pos = _starts(s, T)
        left = (s["offsets"][1:] - s["offsets"][:-1])[seq] - pos     # rows from here to the sequence's end
        row = torch.arange(T, device=x.device)
        dx = torch.zeros(T, C, device=x.device)
        dst = torch.zeros(B, K - 1, C, device=x.device)
        for k in range(K):
            ahead = K - 1 - k
            dx += torch.where((left > ahead)[:, None], dp[(row + ahead).clamp(max=T - 1)] * w[:, k],
                              torch.zeros_like(dx))
            for q in range(ahead):          # the row at position q takes its tap k from state row q + k
                at = (pos == q).nonzero()[:, 0]
                dst[seq[at], q + k] += dp[at] * w[:, k]
    return {"dx": dx.to(x.dtype), "dweight": dw, "dbias": db,
            "dstate0": None if s["state0"] is None else dst.to(x.dtype)}


BLOCK = 64


def _scan_terms(s, lo, hi):
    """Tokens lo..hi of the scan with the token axis first: the step d, the
    decay a [t, b, c, n], the input term, B and C spread over the channels."""
    tok = (lambda v: v[lo:hi, None]) if s["offsets"] is not None else (lambda v: v[:, lo:hi].transpose(0, 1))
    x, raw = tok(s["x"]).float(), tok(s["dt"]).float() + s["dt_bias"]
    d = _softplus(raw)
    rep = s["case"]["C"] // s["case"]["G"]
    Bt = tok(s["Bt"]).float().repeat_interleave(rep, 2)
    Ct = tok(s["Ct"]).float().repeat_interleave(rep, 2)
    a = torch.exp(d[..., None] * s["A"])
    return x, raw, d, a, Bt, Ct, tok


def _plain_scan_states(s, keep):
    """h after every token, block by block: yields (lo, hi, terms, states,
    states before), and leaves the final states in s under `keep`."""
    c = s["case"]
    packed = s["offsets"] is not None
    T, rows = c["T"], 1 if packed else c["B"]
    dev = s["x"].device
    zero = torch.zeros(rows, c["C"], c["N"], device=dev)
    h0 = s.get("h0")
    h = zero if packed or h0 is None else h0
    final = (torch.zeros(c["B"], c["C"], c["N"], device=dev) if h0 is None else h0.clone()) if packed else None
    begins, ends = {}, {}
    if packed:
        for b in range(c["B"]):
            if s["offs"][b + 1] > s["offs"][b]:
                begins[s["offs"][b]] = b
                ends[s["offs"][b + 1] - 1] = b
    for lo in range(0, T, BLOCK):
        hi = min(T, lo + BLOCK)
        terms = _scan_terms(s, lo, hi)
        x, _, d, a, Bt, _, _ = terms
        hs = (d * x)[..., None] * Bt
        before = torch.empty_like(hs)
        for i in range(hi - lo):
            if lo + i in begins:
                h = zero if h0 is None else h0[begins[lo + i]][None]
            before[i] = h
            hs[i].addcmul_(a[i], h)
            h = hs[i]
            if lo + i in ends:
                final[ends[lo + i]] = h[0]
        h = h.clone()
        yield lo, hi, terms, hs, before
    s[keep] = final if packed else h.clone()


def _scan_out(s, x, hs, Ct, tok):
    y = (hs * Ct).sum(-1) + s["skip"] * x
    if s["z"] is None:
        return y, y
    z = tok(s["z"]).float()
    return y, y * z * torch.sigmoid(z)


def _join(s, blocks, dtype):
    v = torch.cat(blocks).to(dtype)
    return v[:, 0].contiguous() if s["offsets"] is not None else v.transpose(0, 1).contiguous()


def _plain_scan(s):
    out = []
    for _, _, (x, _, _, _, _, Ct, tok), hs, _ in _plain_scan_states(s, "last"):
        out.append(_scan_out(s, x, hs, Ct, tok)[1].to(s["x"].dtype))
    return _join(s, out, s["x"].dtype), s.pop("last")


def _plain_scan_step(s):
    c = s["case"]
    x = s["x"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    rep = c["C"] // c["G"]
    Bt, Ct = (s[n].float().repeat_interleave(rep, 1) for n in ("Bt", "Ct"))
    h = s["state"]
    h.copy_(torch.exp(d[..., None] * s["A"]) * h + (d * x)[..., None] * Bt)
    y = (h * Ct).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(s["x"].dtype), h


def _plain_scan_train(s):
    c, dt_ = s["case"], s["x"].dtype
    packed = s["offsets"] is not None
    T, C, N, G = c["T"], c["C"], c["N"], c["G"]
    dev = s["x"].device
    out, first = [], []
    for _, _, (x, _, _, _, _, Ct, tok), hs, before in _plain_scan_states(s, "last"):
        out.append(_scan_out(s, x, hs, Ct, tok)[1].to(dt_))
        first.append(before[0].clone())
    s.pop("last")
    begins = set(s["offs"]) if packed else set()
    dA, dskip, dbias = (torch.zeros(*n, device=dev) for n in ((C, N), (C,), (C,)))
    parts = {n: [] for n in ("dx", "ddt", "dBt", "dCt", "dz")}
    carry = None
    for j in range(len(first) - 1, -1, -1):
        lo, hi = j * BLOCK, min(T, (j + 1) * BLOCK)
        x, raw, d, a, Bt, Ct, tok = _scan_terms(s, lo, hi)
        hs = (d * x)[..., None] * Bt
        before = torch.empty_like(hs)
        h = first[j]
        for i in range(hi - lo):
            if lo + i in begins:
                h = torch.zeros_like(h)
            before[i] = h
            hs[i].addcmul_(a[i], h)
            h = hs[i]
        dy = tok(s["dy"]).float()
        if s["z"] is not None:
            z = tok(s["z"]).float()
            sg = torch.sigmoid(z)
            y = (hs * Ct).sum(-1) + s["skip"] * x
            parts["dz"].append((dy * y * sg * (1 + z * (1 - sg))).to(dt_))
            dy = dy * z * sg
        gr = dy[..., None] * Ct                # gradient of h_t, the later tokens' share added below
        dCt = dy[..., None] * hs
        if carry is not None:
            gr[-1] += carry
        for i in range(hi - lo - 2, -1, -1):
            if lo + i + 1 not in begins:
                gr[i].addcmul_(a[i + 1], gr[i + 1])
        carry = torch.zeros_like(gr[0]) if lo in begins else a[0] * gr[0]
        du = (gr * Bt).sum(-1)
        dBt = gr * (d * x)[..., None]
        q = gr * before * a
        dd = (du * x + (q * s["A"]).sum(-1)) * torch.sigmoid(raw)
        dA += (q * d[..., None]).sum((0, 1))
        dskip += (dy * x).sum((0, 1))
        dbias += dd.sum((0, 1))
        parts["dx"].append((du * d + s["skip"] * dy).to(dt_))
        parts["ddt"].append(dd.to(dt_))
        for n, v in (("dBt", dBt), ("dCt", dCt)):
            parts[n].append(v.unflatten(2, (G, C // G)).sum(3).to(dt_))
    g = {n: _join(s, v[::-1], dt_) if v else None for n, v in parts.items()}
    g.update(dA=dA, dskip=dskip, ddt_bias=dbias, dh0=None)
    return _join(s, out, dt_), g


def _plain_norm_parts(s):
    x = s["x"].float()
    if s["case"]["kind"] == "layer":
        x = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    xh = x * r
    n = xh * s["weight"]
    return xh, r, n if s["bias"] is None else n + s["bias"]


def _plain_norm(s):
    _, _, n = _plain_norm_parts(s)
    if s["z"] is not None:
        z = s["z"].float()
        n = n * z * torch.sigmoid(z)
    return n.to(s["x"].dtype)


def _plain_norm_backward(s):
    xh, r, n = _plain_norm_parts(s)
    dy, dz = s["dy"].float(), None
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        dz = (dy * n * sg * (1 + z * (1 - sg))).to(s["x"].dtype)
        dy = dy * z * sg
    dw, db = (dy * xh).sum(0), dy.sum(0)
    v = dy * s["weight"]
    dx = v - xh * (v * xh).mean(1, keepdim=True)
    if s["case"]["kind"] == "layer":
        dx = dx - v.mean(1, keepdim=True)
    return {"dx": (dx * r).to(s["x"].dtype), "dweight": dw, "dbias": None if s["bias"] is None else db, "dz": dz}


_PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv_step, "conv_backward": _plain_conv_backward,
          "scan": _plain_scan, "scan_step": _plain_scan_step, "scan_train": _plain_scan_train, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _f64(s):
    return {n: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for n, v in s.items()}


def _sequences(s):
    """Each sequence's rows: an index into a dense batch, or a slice of the packed rows."""
    if s.get("offsets") is None:
        return [(b,) for b in range(s["case"]["B"])]
    return [slice(s["offs"][b], s["offs"][b + 1]) for b in range(s["case"]["B"])]


def _silu_slope(v):
    e = torch.exp(-v)
    return (1 + e + v * e) / (1 + e) ** 2


def _exact_conv(s, backward):
    w, bias, K = s["weight"], s["bias"], s["weight"].shape[1]
    y = torch.zeros(s["x"].shape, dtype=torch.float64, device=w.device)
    states, dstates = [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b, at in enumerate(_sequences(s)):
        x = s["x"][at]
        old = torch.zeros(K - 1, w.shape[0], dtype=torch.float64, device=w.device) if s["state0"] is None \
            else s["state0"][b]
        rows = torch.cat([old, x])
        win = torch.stack([rows[k:k + x.shape[0]] for k in range(K)], 2)     # [t, c, k]
        p = torch.einsum("tck,ck->tc", win, w) + bias
        if not backward:
            y[at] = p / (1 + torch.exp(-p))
            states.append(rows[x.shape[0]:])
            continue
        dp = s["dy"][at] * _silu_slope(p)
        dw += torch.einsum("tc,tck->ck", dp, win)
        db += dp.sum(0)
        full = torch.zeros(x.shape[0] + K - 1, w.shape[0], dtype=torch.float64, device=w.device)
        for t in range(K):
            full[t:t + x.shape[0]] += dp * w[:, t]
        y[at] = full[K - 1:]
        dstates.append(full[:K - 1])
    if not backward:
        return y, torch.stack(states)
    return {"dx": y, "dweight": dw, "dbias": db, "dstate0": None if s["state0"] is None else torch.stack(dstates)}


def _exact_step(s, x, dt, Bt, Ct, h):
    """One token: (y before the gate, h, decay, step, raw step, B and C per channel)."""
    G, C = s["case"]["G"], s["case"]["C"]
    raw = dt + s["dt_bias"]
    d = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    wide = lambda v: v[..., :, None, :].expand(*v.shape[:-2], G, C // G, v.shape[-1]).reshape(  # noqa: E731
        *v.shape[:-2], C, v.shape[-1])
    Bc, Cc = wide(Bt), wide(Ct)
    a = torch.exp(d.unsqueeze(-1) * s["A"])
    h = a * h + d.unsqueeze(-1) * x.unsqueeze(-1) * Bc
    return torch.einsum("...cn,...cn->...c", h, Cc) + s["skip"] * x, h, a, d, raw, Bc, Cc


def _runs(s):
    """Independent runs of tokens: the whole dense batch at once, or one packed sequence at a time."""
    if s.get("offsets") is None:
        yield slice(None), lambda v, t: v[:, t], s["case"]["T"]
        return
    for b in range(s["case"]["B"]):
        lo, hi = s["offs"][b], s["offs"][b + 1]
        yield slice(b, b + 1), lambda v, t, lo=lo: v[lo + t][None], hi - lo


def _exact_scan(s, backward=False):
    c, dev = s["case"], s["x"].device
    h_all = torch.zeros(c["B"], c["C"], c["N"], dtype=torch.float64, device=dev) if s.get("h0") is None \
        else s["h0"].clone()
    new = lambda n: torch.zeros(s[n].shape, dtype=torch.float64, device=dev)  # noqa: E731
    y = new("x")
    g = {"dx": new("x"), "ddt": new("dt"), "dBt": new("Bt"), "dCt": new("Ct"),
         "dz": None if s["z"] is None else new("z"), "dA": new("A"), "dskip": new("skip"),
         "ddt_bias": new("dt_bias"), "dh0": None} if backward else None
    for rows, tok, count in _runs(s):
        h = h_all[rows].clone()
        past = [h]
        for t in range(count):
            v, h, *_ = _exact_step(s, *(tok(s[n], t) for n in ("x", "dt", "Bt", "Ct")), h)
            if s["z"] is not None:
                z = tok(s["z"], t)
                v = v * z / (1 + torch.exp(-z))
            tok(y, t).copy_(v)
            if backward:
                past.append(h)
        h_all[rows] = h
        if not backward:
            continue
        lam = torch.zeros_like(h)
        for t in range(count - 1, -1, -1):
            x = tok(s["x"], t)
            v, h, a, d, raw, Bc, Cc = _exact_step(s, x, *(tok(s[n], t) for n in ("dt", "Bt", "Ct")), past[t])
            dy = tok(s["dy"], t)
            if s["z"] is not None:
                z = tok(s["z"], t)
                tok(g["dz"], t).copy_(dy * v * _silu_slope(z))
                dy = dy * z / (1 + torch.exp(-z))
            lam = lam + dy.unsqueeze(-1) * Cc
            du = (lam * Bc).sum(-1)
            decay = lam * a * past[t]
            dd = (du * x + (decay * s["A"]).sum(-1)) / (1 + torch.exp(-raw))
            tok(g["dx"], t).copy_(du * d + dy * s["skip"])
            tok(g["ddt"], t).copy_(dd)
            for n, val in (("dBt", lam * (d * x).unsqueeze(-1)), ("dCt", dy.unsqueeze(-1) * h)):
                to = tok(g[n], t)
                to.copy_(val.reshape(val.shape[0], c["G"], -1, c["N"]).sum(2))
            g["dA"] += (decay * d.unsqueeze(-1)).sum(0)
            g["dskip"] += (dy * x).sum(0)
            g["ddt_bias"] += dd.sum(0)
            lam = a * lam
    return (y, g) if backward else (y, h_all)


def _exact_norm(s, backward):
    x, w = s["x"], s["weight"]
    bias = 0.0 if s["bias"] is None else s["bias"]
    centre = s["case"]["kind"] == "layer"
    m = x.mean(1, keepdim=True) if centre else torch.zeros_like(x[:, :1])
    sd = ((x - m).square().mean(1, keepdim=True) + EPS).sqrt()
    n = (x - m) / sd * w + bias
    gate = 1.0 if s["z"] is None else s["z"] / (1 + torch.exp(-s["z"]))
    if not backward:
        return n * gate
    dn = s["dy"] * gate
    dxh = dn * w
    # through the division by sd, then through the mean
    dcen = dxh / sd - (x - m) * (dxh * (x - m)).sum(1, keepdim=True) / (x.shape[1] * sd ** 3)
    dx = dcen - dcen.mean(1, keepdim=True) if centre else dcen
    return {"dx": dx, "dweight": (dn * (x - m) / sd).sum(0), "dbias": None if s["bias"] is None else dn.sum(0),
            "dz": None if s["z"] is None else s["dy"] * n * _silu_slope(s["z"])}


def exact(case, seed):
    s = _f64(prepare(case, seed))
    op = case["op"]
    if op in ("conv", "conv_backward"):
        return _exact_conv(s, op == "conv_backward")
    if op == "conv_step":
        rows = torch.cat([s["state"], s["x"].unsqueeze(1)], 1)
        p = torch.einsum("bkc,ck->bc", rows, s["weight"]) + s["bias"]
        return p / (1 + torch.exp(-p)), rows[:, 1:]
    if op == "scan":
        return _exact_scan(s)
    if op == "scan_train":
        return _exact_scan(s, True)
    if op == "scan_step":
        y, h, *_ = _exact_step(s, s["x"], s["dt"], s["Bt"], s["Ct"], s["state"])
        return y if s["z"] is None else y * s["z"] / (1 + torch.exp(-s["z"])), h
    return _exact_norm(s, op == "norm_backward")


def work(case):
    e, op, C = (2 if case["dtype"] == "bf16" else 4), case["op"], case["C"]
    if op in ("norm", "norm_backward"):
        n = case["R"] * C
        arrays = (2 + case["gate"]) if op == "norm" else (3 + 2 * case["gate"])
        params = C * 4 * ((1 if op == "norm" else 2) * (2 if case["kind"] == "layer" else 1))
        return {"bytes": n * e * arrays + params, "flops": n * (8 if op == "norm" else 16)}
    B = case["B"]
    if op.startswith("conv"):
        K = case["K"]
        state = B * (K - 1) * C * e
        if op == "conv_step":
            return {"bytes": 2 * B * C * e + 2 * state + C * (K + 1) * 4, "flops": B * C * (2 * K + 5)}
        n = (case["T"] if case["packed"] else B * case["T"]) * C
        if op == "conv":
            return {"bytes": 2 * n * e + state * (1 + case["init"]) + C * (K + 1) * 4, "flops": n * (2 * K + 5)}
        return {"bytes": 3 * n * e + 2 * state * case["init"] + 2 * C * (K + 1) * 4, "flops": n * (6 * K + 12)}
    N, G = case["N"], case["G"]
    params = C * (N + 2) * 4
    if op == "scan_step":
        return {"bytes": B * (C * (3 + case["gate"]) + 2 * G * N) * e + 2 * B * C * N * 4 + params,
                "flops": B * C * (7 * N + 12)}
    rows = case["T"] if case["packed"] else B * case["T"]
    state = B * C * N * 4
    if op == "scan":
        return {"bytes": rows * (C * (3 + case["gate"]) + 2 * G * N) * e + state * (1 + case["init"]) + params,
                "flops": rows * C * (7 * N + 12)}
    # forward and backward: x, dt, B, C (and z) in, y out; then those and dy in, their gradients out
    return {"bytes": rows * (C * (3 + case["gate"]) + 2 * G * N) * e + rows * (C * (5 + 2 * case["gate"]) + 4 * G * N) * e
            + 3 * params, "flops": rows * C * (25 * N + 30)}
