// gdr2_glr_backward.hip -- gradients of the gated linear recurrence.
//
// With s the logistic sigmoid, q = sqrt(1 - a^2) and g_t = dL/dh_t:
//   g_t = dy_t + a_{t+1} g_{t+1} (dL/dh_out behind the last token)
//   dx = g q s(i),  di = g q x s(i) (1 - s(i))
//   du = g (a h_{t-1} - s(i) x a^2 / q),  dr = du A s(r) (1 - s(r)),  dA = sum du s(r)
//   dL/dh0 = a_1 g_1
// The recurrence of g runs backwards over the layout of gdr2_glr.h: a
// sub-chunk maps the gradient that reaches it from behind, lam = a g of the
// token after it, to the one it hands on, lam -> P lam + L.  The states within a sub-chunk
// are formed again from the recorded one before its first token, so nothing
// runs forwards over the sequence.
//
// 14 bytes an element of bf16 rows (9 of rows in 8 bits) and 0.25 of recorded states.
#include <algorithm>
#include <type_traits>

#include "gdr2_glr.h"

namespace gdr2 {

namespace {

// ---- rows in 8 bits --------------------------------------------------------
// A sub-chunk's codes; lane k of a block's lanes holds the scale of token k.
template <int V> struct SubCodes {
    uint32_t raw[kGlrChunk];
    uint32_t scale[V == 1 ? kGlrChunk : 1];

    template <typename R, typename S>
    __device__ __forceinline__ void load(R codes, uint32_t off, uint32_t row_bytes, S scales, uint32_t soff, uint32_t scale_bytes,
                                         bool full)
    {
        for_tokens(full, off, row_bytes, [&](int k, uint32_t at, uint32_t row) {
            if constexpr (V == 2)
                raw[k] = __builtin_amdgcn_raw_buffer_load_b16(codes, at, row, 0);
            else
                raw[k] = __builtin_amdgcn_raw_buffer_load_b8(codes, at, row, 0);
        });
        if constexpr (V == 2) {
            // 16 lanes hold a block, as many as a sub-chunk has tokens
            static_assert(kRows8 / V == kGlrChunk, "one lane a token");
            scale[0] = __builtin_amdgcn_raw_buffer_load_b8(scales, soff + (threadIdx.x % kGlrChunk) * scale_bytes, 0, 0);
        } else {
            for_tokens(full, soff, scale_bytes, [&](int k, uint32_t at, uint32_t row) {
                scale[k] = __builtin_amdgcn_raw_buffer_load_b8(scales, at, row, 0);
            });
        }
    }
    template <int K> __device__ __forceinline__ void token(float (&v)[V]) const
    {
        Codes<V> c;
        c.w[0] = raw[K];
        if constexpr (V == 2)
            c.get(__builtin_amdgcn_update_dpp(0, scale[0], 0x150 + K, 0xF, 0xF, true), v);   // row_newbcast
        else
            c.get(scale[K], v);
    }
};

// The sub-chunk's x, r and i, from rows or from codes.
template <typename T, int V, bool P8> struct GradInputs;
template <typename T, int V> struct GradInputs<T, V, false> {
    SubRows<T, V> x, r, i;
};
template <typename T, int V> struct GradInputs<T, V, true> {
    SubCodes<V> x, r, i;
};
template <int K, typename T, int V> __device__ __forceinline__ void token_of(const SubRows<T, V>& s, float (&v)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j)
        v[j] = s.get(K, j);
}
template <int K, int V> __device__ __forceinline__ void token_of(const SubCodes<V>& s, float (&v)[V]) { s.template token<K>(v); }

// f(0) .. f(15), the token's number a constant (DPP's broadcast lane is an immediate)
template <int K = 0, typename F> __device__ __forceinline__ void tokens_up(const F& f)
{
    if constexpr (K < kGlrChunk) {
        f(std::integral_constant<int, K>());
        tokens_up<K + 1>(f);
    }
}

// Where an array's rows lie, for the wave's rows of a tile.
struct Source {
    WaveRows rows, scales;
    uint32_t off, soff;
    template <typename T, int V, int LR>
    static __device__ __forceinline__ Source of_rows(const void* p, int64_t row0, int64_t ld, const GlrLane<V, LR>& lane)
    {
        Source s{};
        s.rows = WaveRows::at<T>(p, row0, ld);
        s.off = lane.template offset<T>(s.rows.row_bytes);
        return s;
    }
    template <int V, int LR>
    static __device__ __forceinline__ Source of_codes(const gdr2_rows8& p, int64_t row0, int64_t C, const GlrLane<V, LR>& lane)
    {
        Source s{};
        s.rows = WaveRows::at<uint8_t>(p.codes, row0, C);
        s.scales = WaveRows::at<uint8_t>(p.scales, row0, scale_count(C));
        s.off = lane.template offset<uint8_t>(s.rows.row_bytes);
        s.soff = lane.scale_offset(s.scales.row_bytes, C);
        return s;
    }
    template <typename T, int V> __device__ __forceinline__ void load(SubRows<T, V>& to, int64_t at, int left, bool full) const
    {
        to.load(rows.buffer(at, left), off, rows.row_bytes, full);
    }
    template <int V> __device__ __forceinline__ void load(SubCodes<V>& to, int64_t at, int left, bool full) const
    {
        to.load(rows.buffer(at, left), off, rows.row_bytes, scales.buffer(at, left), soff, scales.row_bytes, full);
    }
};

// The gradient that reaches the segment's end: dL/dh_out, and the segments
// behind it in turn, the last one first.
template <int V>
__device__ __forceinline__ void end_gradient(const float* dh_out, const float* spans, const Piece& q, int64_t count, int64_t C,
                                             int64_t c, bool on, float (&lam)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        lam[v] = 0.f;
    if (!on)
        return;
    if (dh_out)
        load_channels<V>(dh_out + q.seq * C + c, lam);
    const float* s = spans + (q.first * C + c) * 2;
    for (int64_t j = count - 1; j > q.index; j -= kFoldAhead) {
        float pl[kFoldAhead][2 * V];
#pragma unroll
        for (int u = 0; u < kFoldAhead; ++u)
            if (j - u > q.index)
                load_channels<2 * V>(s + (j - u) * C * 2, pl[u]);
#pragma unroll
        for (int u = 0; u < kFoldAhead; ++u)
            if (j - u > q.index)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    lam[v] = fmaf(pl[u][2 * v], lam[v], pl[u][2 * v + 1]);
    }
}

// A sub-chunk's (P, L) through LDS: the gradient that reaches this lane's
// sub-chunk from behind, and in `lam` the one that leaves the tile.
template <int V, int LR, bool SPAN>
__device__ __forceinline__ void reverse_fold(const float (*s_span)[LR][2 * V], const GlrLane<V, LR>& lane, float (&lam)[V],
                                             float (&reach)[V], float (&whole)[V])
{
#pragma unroll
    for (int j = GlrTile<LR>::kSubs - 1; j >= 0; --j) {
        float pl[2 * V];
#pragma unroll
        for (int v = 0; v < 2 * V; ++v)
            pl[v] = s_span[j][lane.li][v];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            reach[v] = j == lane.sub || j == GlrTile<LR>::kSubs - 1 ? lam[v] : reach[v];
            lam[v] = fmaf(pl[2 * v], lam[v], pl[2 * v + 1]);
            if constexpr (SPAN)
                whole[v] *= pl[2 * v];
        }
        if (j % 8 == 0)
            __builtin_amdgcn_sched_barrier(0);       // eight reads in flight at most
    }
}

template <int V, int LR> struct TileRows {
    int64_t n;
    int wave;
    __device__ __forceinline__ int64_t first(int64_t t) const { return t + wave * GlrTile<LR>::kWaveTokens; }
    __device__ __forceinline__ int left(int64_t t) const
    {
        constexpr int W = GlrTile<LR>::kWaveTokens;
        const int64_t m = t < 0 ? 0 : n - first(t);
        return (int)(m < 0 ? 0 : m > W ? W : m);
    }
};

// (P, L) of every segment but a sequence's first one.
template <typename T, int V, int LR, bool P8>
__global__ __launch_bounds__(64 * kGlrWaves) void glr_span_backward_kernel(gdr2_glr_bwd_args p, GlrPlan plan, float* spans)
{
    typedef GlrTile<LR> Tile;
    __shared__ float s_span[2][Tile::kSubs][LR][2 * V];
    const gdr2_glr_args& a = p.f;
    const int64_t slot = blockIdx.x / plan.blocks, block = blockIdx.x - slot * plan.blocks;
    const Segment seg = segment_of(plan, slot);
    if (seg.q.seq < 0 || seg.q.index == 0)
        return;
    const GlrLane<V, LR> lane(a.C, block);
    const int64_t row0 = seg.q.row0 + seg.t0;
    const TileRows<V, LR> rows{seg.n, lane.wave};
    const Source sr = P8 ? Source::of_codes<V, LR>(a.r8, row0, a.C, lane) : Source::of_rows<T, V, LR>(a.r, row0, a.r_stride, lane);
    const Source sd = Source::of_rows<T, V, LR>(p.dy, row0, a.C, lane);
    float A2[V], lam[V], whole[V], reach[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A2[v] = lane.on ? exponent_scale(a.A[lane.c + v]) : 0.f;
        lam[v] = 0.f;
        whole[v] = 1.f;
    }
    auto fetch = [&](decltype(GradInputs<T, V, P8>::r)& r, SubRows<T, V>& dy, int64_t t) {
        const int m = rows.left(t);
        const int64_t at = m > 0 ? rows.first(t) : 0;
        sr.load(r, at, m, m == Tile::kWaveTokens);
        sd.load(dy, at, m, m == Tile::kWaveTokens);
    };
    decltype(GradInputs<T, V, P8>::r) next_r;
    SubRows<T, V> next_dy;
    const int64_t last = (seg.n - 1) / Tile::kTokens * Tile::kTokens;
    fetch(next_r, next_dy, last);
    int buf = 0;
    for (int64_t t = last; t >= 0; t -= Tile::kTokens, buf ^= 1) {
        const auto r = next_r;
        const SubRows<T, V> dy = next_dy;
        fetch(next_r, next_dy, t - Tile::kTokens);
        const int mine = rows.left(t) - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
        float at[kGlrChunk][V], P[V], L[V];
        tokens_up([&](auto at_k) {
                constexpr int K = decltype(at_k)::value;
            float rv[V];
            token_of<K>(r, rv);
#pragma unroll
            for (int v = 0; v < V; ++v)
                at[K][v] = __builtin_unpredictable(K < mine) ? fast_exp2(A2[v] * sigmoid_f(rv[v])) : 1.f;
        });
#pragma unroll
        for (int v = 0; v < V; ++v) {
            P[v] = 1.f;
            L[v] = 0.f;
        }
#pragma unroll
        for (int k = kGlrChunk - 1; k >= 0; --k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                L[v] = at[k][v] * (dy.get(k, v) + L[v]);
                P[v] *= at[k][v];
            }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_span[buf][lane.sub][lane.li][2 * v] = P[v];
            s_span[buf][lane.sub][lane.li][2 * v + 1] = L[v];
        }
        lds_barrier();
        reverse_fold<V, LR, true>(s_span[buf], lane, lam, reach, whole);
    }
    if (lane.sub != 0 || !lane.on)
        return;
    float* to = spans + (slot * a.C + lane.c) * 2;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        to[2 * v] = whole[v];
        to[2 * v + 1] = lam[v];
    }
}

template <typename T, int V, int LR, bool P8>
__global__ __launch_bounds__(64 * kGlrWaves) void glr_backward_kernel(gdr2_glr_bwd_args p, GlrPlan plan, const float* spans, float* part)
{
    typedef GlrTile<LR> Tile;
    __shared__ float s_span[2][Tile::kSubs][LR][2 * V];
    const gdr2_glr_args& a = p.f;
    const int64_t slot = blockIdx.x / plan.blocks, block = blockIdx.x - slot * plan.blocks;
    const Segment seg = segment_of(plan, slot);
    const GlrLane<V, LR> lane(a.C, block);
    float dA[V], A2[V], Av[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Av[v] = lane.on ? finite(a.A[lane.c + v]) : 0.f;
        A2[v] = exponent_scale(Av[v]);
        dA[v] = 0.f;
    }
    if (seg.q.seq >= 0) {
        const int64_t row0 = seg.q.row0 + seg.t0;
        const TileRows<V, LR> rows{seg.n, lane.wave};
        Source sx, sr, si;
        if constexpr (P8) {
            sx = Source::of_codes<V, LR>(a.x8, row0, a.C, lane);
            sr = Source::of_codes<V, LR>(a.r8, row0, a.C, lane);
            si = Source::of_codes<V, LR>(a.i8, row0, a.C, lane);
        } else {
            sx = Source::of_rows<T, V, LR>(a.x, row0, a.x_stride, lane);
            sr = Source::of_rows<T, V, LR>(a.r, row0, a.r_stride, lane);
            si = Source::of_rows<T, V, LR>(a.i, row0, a.i_stride, lane);
        }
        const Source sd = Source::of_rows<T, V, LR>(p.dy, row0, a.C, lane);
        const WaveRows ox = WaveRows::at<T>(p.dx, row0, a.C), orr = WaveRows::at<T>(p.dr, row0, a.C), oi = WaveRows::at<T>(p.di, row0, a.C);
        const uint32_t off = lane.template offset<T>(ox.row_bytes);
        const int64_t chunk0 = chunk_row(a, seg.q) + seg.t0 / kGlrChunk;
        const int64_t L = (int64_t)1 << plan.seg.lg, count = plan.split ? (seg.q.len + L - 1) >> plan.seg.lg : 1;
        float lam[V], reach[V], unused[V];
        end_gradient<V>(p.dh_out, spans, seg.q, count, a.C, lane.c, lane.on, lam);

        // r, dy and the recorded state of the next tile are on their way through the second half of this one, x and i
        // of this one through its first half
        decltype(GradInputs<T, V, P8>::r) r;
        SubRows<T, V> dy;
        float h0[V];
        auto fetch = [&](int64_t t) {
            const int m = rows.left(t), mine = m - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
            const int64_t at = m > 0 ? rows.first(t) : 0;
            sr.load(r, at, m, m == Tile::kWaveTokens);
            sd.load(dy, at, m, m == Tile::kWaveTokens);
#pragma unroll
            for (int v = 0; v < V; ++v)
                h0[v] = 0.f;
            if (lane.on && mine > 0)
                load_channels<V>(a.h_chunks + (chunk0 + t / kGlrChunk + lane.sub) * a.C + lane.c, h0);
        };
        const int64_t last = seg.n > 0 ? (seg.n - 1) / Tile::kTokens * Tile::kTokens : -1;
        if (last >= 0)
            fetch(last);
        int buf = 0;
        for (int64_t t = last; t >= 0; t -= Tile::kTokens, buf ^= 1) {
            const int left = rows.left(t), mine = left - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
            const int64_t first = left > 0 ? rows.first(t) : 0;
            decltype(GradInputs<T, V, P8>::x) x, i;
            sx.load(x, first, left, left == Tile::kWaveTokens);
            si.load(i, first, left, left == Tile::kWaveTokens);
            float at[kGlrChunk][V], sg[kGlrChunk][V], g[kGlrChunk][V], P[V], Lr[V];
            tokens_up([&](auto at_k) {
                constexpr int K = decltype(at_k)::value;
                float rv[V];
                token_of<K>(r, rv);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    sg[K][v] = sigmoid_f(rv[v]);
            });
            if (left < Tile::kWaveTokens) {
#pragma unroll
                for (int k = 0; k < kGlrChunk; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        sg[k][v] = k < mine ? sg[k][v] : 0.f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                P[v] = 1.f;
                Lr[v] = 0.f;
            }
#pragma unroll
            for (int k = kGlrChunk - 1; k >= 0; --k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    at[k][v] = fast_exp2(A2[v] * sg[k][v]);
                    Lr[v] = at[k][v] * (dy.get(k, v) + Lr[v]);
                    P[v] *= at[k][v];
                }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s_span[buf][lane.sub][lane.li][2 * v] = P[v];
                s_span[buf][lane.sub][lane.li][2 * v + 1] = Lr[v];
            }
            lds_barrier();
            reverse_fold<V, LR, false>(s_span[buf], lane, lam, reach, unused);
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = h0[v];
#pragma unroll
            for (int k = kGlrChunk - 1; k >= 0; --k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    g[k][v] = dy.get(k, v) + reach[v];
                    reach[v] = at[k][v] * g[k][v];
                }
            __builtin_amdgcn_sched_barrier(0);
            const auto bx = ox.buffer(first, left), br = orr.buffer(first, left), bi = oi.buffer(first, left);
            // a token's row in the lanes' or in the scalar offset, as for_tokens places it
            const bool full = left == Tile::kWaveTokens;
            uint32_t row_bytes = ox.row_bytes;
            asm volatile("" : "+s"(row_bytes));
            tokens_up([&](auto at_k) {
                constexpr int K = decltype(at_k)::value;
                float xv[V], iv[V], dx[V], dr[V], di[V];
                token_of<K>(x, xv);
                token_of<K>(i, iv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float s = sg[K][v], e = at[K][v], q = glr_root(A2[v] * s, e);
                    // a masked token's x and i have no part, whatever they hold
                    const float all = sigmoid_f(iv[v]), o = unless_masked(q, all), in = unless_masked(q, all * xv[v]);
                    const float gq = g[K][v] * q;
                    dx[v] = gq * o;
                    di[v] = gq * in * (1.f - o);
                    // 1/q where q is 0: anything finite, for `in` is 0
                    const float over = e * e * __builtin_amdgcn_rcpf(fmaxf(q, 1e-30f));
                    const float du = g[K][v] * fmaf(e, h[v], -in * over);
                    dA[v] = fmaf(du, s, dA[v]);
                    dr[v] = du * (Av[v] * fmaf(-s, s, s));
                    h[v] = fmaf(e, h[v], q * in);
                }
                const uint32_t row = K * row_bytes, lane_row = full ? off : off + row, all_row = full ? row : 0;
                store_token<T, V>(bx, lane_row, all_row, dx);
                store_token<T, V>(br, lane_row, all_row, dr);
                store_token<T, V>(bi, lane_row, all_row, di);
                // tokens are scheduled four at a time, and the next tile's loads take the registers of the first half:
                // more in flight would not fit
                if constexpr (K % 4 == 3)
                    __builtin_amdgcn_sched_barrier(0);
                if constexpr (K == kGlrChunk / 2 - 1)
                    fetch(t - Tile::kTokens);
            });
        }
        if (p.dh0 && seg.q.index == 0 && lane.sub == 0 && lane.on)
            store_channels<V>(p.dh0 + seg.q.seq * a.C + lane.c, lam);
    }
    // dA over the workgroup's sub-chunks, in their order; an idle slot's are 0
    float (*s_sum)[LR][V] = reinterpret_cast<float (*)[LR][V]>(&s_span[0][0][0][0]);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
        s_sum[lane.sub][lane.li][v] = dA[v];
    __syncthreads();
    if (lane.sub == 0 && lane.on) {
        for (int j = 1; j < Tile::kSubs; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v)
                dA[v] += s_sum[j][lane.li][v];
        store_channels<V>(part + slot * a.C + lane.c, dA);
    }
}

int64_t span_floats(const gdr2_glr_args& a, const GlrPlan& p) { return p.split ? p.seg.slots() * a.C * 2 : 0; }

template <typename T, int V, int LR, bool P8>
hipError_t backward_lr(const gdr2_glr_bwd_args& p, const GlrPlan& plan, hipStream_t stream)
{
    const dim3 grid((unsigned)(plan.seg.slots() * plan.blocks)), threads(64 * kGlrWaves);
    float* spans = (float*)p.workspace;
    float* part = spans + span_floats(p.f, plan);
    const int64_t P = p.f.B > 0 ? plan.seg.slots() : 0;
    if (P > 0) {
        if (plan.split) {
            hipLaunchKernelGGL((glr_span_backward_kernel<T, V, LR, P8>), grid, threads, 0, stream, p, plan, spans);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess)
                return e;
        }
        hipLaunchKernelGGL((glr_backward_kernel<T, V, LR, P8>), grid, threads, 0, stream, p, plan, spans, part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return launch_column_sum(part, P, p.f.C, {p.dA, p.f.C}, {nullptr, 0}, {nullptr, 0}, stream);
}

template <bool P8> hipError_t backward_p(const gdr2_glr_bwd_args& p, hipStream_t stream)
{
    if (glr_pairs(p.f)) {
        const GlrPlan plan = glr_plan(p.f, 2, true);
        return plan.lr == 32 ? backward_lr<bf16, 2, 32, P8>(p, plan, stream) : backward_lr<bf16, 2, 16, P8>(p, plan, stream);
    }
    const GlrPlan plan = glr_plan(p.f, 1, true);
    return p.f.dtype == GDR2_BF16 ? backward_lr<bf16, 1, 64, P8>(p, plan, stream) : backward_lr<float, 1, 64, P8>(p, plan, stream);
}

}  // namespace

// The larger of the two widths' needs where the pointers decide between them.
size_t glr_backward_workspace_bytes(const gdr2_glr_bwd_args& p)
{
    int64_t most = 0;
    for (int V : {1, 2}) {
        if (V == 2 && (p.f.C % 2 || p.f.dtype != GDR2_BF16))
            continue;
        const GlrPlan plan = glr_plan(p.f, V, true);
        most = std::max(most, span_floats(p.f, plan) + plan.seg.slots() * p.f.C);
    }
    return p.f.B > 0 ? (size_t)most * sizeof(float) : 0;
}

hipError_t launch_glr_backward(const gdr2_glr_bwd_args& p, hipStream_t stream)
{
    return p.f.x ? backward_p<false>(p, stream) : backward_p<true>(p, stream);
}

int64_t glr_launch_groups(const gdr2_glr_args& a, bool backward)
{
    int64_t most = 0;
    for (int V : {1, 2}) {
        if (V == 2 && (a.C % 2 || a.dtype != GDR2_BF16))
            continue;
        const GlrPlan plan = glr_plan(a, V, backward);
        const double groups = (double)plan.seg.slots() * (double)plan.blocks * (kGlrWaves * 64 / 256);
        most = groups >= (double)kMaxGroups ? kMaxGroups : std::max(most, (int64_t)groups);
    }
    return most;
}

}  // namespace gdr2
