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
// 14 bytes an element of bf16 rows (11.1 from rows in 8 bits) and 0.25 of
// recorded states, 60 vector operations in one pass, 66 in chained tiles (68 from 8
// bits).  8x4096x2048 in chained tiles 224 us (4.3 TB/s; a large copy 5.15): seven
// streams at a time, the vector units busy for 56 % of it.  From 8 bits 4x4096x2048
// 116 us (3.3 TB/s), where waves wait for data for 37 % of their time: 161
// registers leave three of them a SIMD.
#include <algorithm>
#include <type_traits>

#include "gdr2_glr.h"

namespace gdr2 {

namespace {

// ---- rows in 8 bits --------------------------------------------------------
// A sub-chunk's codes; with two channels a lane, lane k of a block's 16 lanes
// holds the scale of token k.
template <int V> struct SubCodes {
    uint32_t raw[kGlrChunk];
    uint32_t scale[V == 1 ? kGlrChunk : 1];
    template <int K> __device__ __forceinline__ void token(float (&v)[V]) const
    {
        if constexpr (V == 2)
            values_of<V>(raw[K], __builtin_amdgcn_update_dpp(0, scale[0], 0x150 + K, 0xF, 0xF, true), v);   // row_newbcast
        else
            values_of<V>(raw[K], scale[K], v);
    }
};

template <int K, typename T, int V> __device__ __forceinline__ void token_of(const SubRows<T, V>& s, float (&v)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j)
        v[j] = s.get(K, j);
}
template <int K, int V> __device__ __forceinline__ void token_of(const SubCodes<V>& s, float (&v)[V]) { s.template token<K>(v); }

// A gate as it is kept between the passes: the smaller of s and 1 - s, with the
// sign of r.  The slope s (1 - s) of an open gate is then as exact as that of a
// closed one; from s alone it lost 1 % at r = 12 and all from 17 on.  The logistic
// comes back as the fraction of -v, -v or 1 - v (at most 1 - 2^-24): one operation,
// and no register more.  r goes in as at most 87, for 0 has the fraction 0;
// -inf gives 0.  (The minimum of a NaN is NaN.)
__device__ __forceinline__ float kept_gate(float r)
{
    const float m = __builtin_elementwise_minimum(r, 87.f), e = fast_exp2(-kLog2e * fabsf(m));
    return copysignf(e * __builtin_amdgcn_rcpf(1.f + e), m);
}
__device__ __forceinline__ float gate_of(float kept) { return __builtin_amdgcn_fractf(-kept); }
__device__ __forceinline__ float gate_slope(float kept) { return fmaf(-kept, kept, fabsf(kept)); }

// f(0) .. f(15), the token's number a constant (DPP's broadcast lane is an immediate)
template <int K = 0, typename F> __device__ __forceinline__ void tokens_up(const F& f)
{
    if constexpr (K < kGlrChunk) {
        f(std::integral_constant<int, K>());
        tokens_up<K + 1>(f);
    }
}

// One array's rows, from the segment's first one on.
template <typename T, int V, bool P8> struct Source {
    typedef SubRows<T, V> Tokens;
    WaveRows rows;
    uint32_t off;
    template <int LR> __device__ __forceinline__ Source(const void* p, int64_t row0, int64_t ld, const GlrLane<V, LR>& lane)
        : rows(WaveRows::at<T>(p, row0, ld)), off(lane.template offset<T>(rows.row_bytes))
    {
    }
    template <int LR>
    __device__ __forceinline__ Source(const void* p, const gdr2_rows8&, int64_t row0, int64_t ld, int64_t, const GlrLane<V, LR>& lane)
        : Source(p, row0, ld, lane)
    {
    }
    // The tokens of one tile, in turn: the wave's first one is `first`, `left` of them exist.
    struct Reader {
        __amdgpu_buffer_rsrc_t rsrc;
        RowOffset at;
        __device__ __forceinline__ void load(int k, Tokens& to) { to.load(k, rsrc, at); }
    };
    __device__ __forceinline__ Reader reader(int64_t first, int left) const { return {rows.buffer(first, left), {off, rows.row_bytes}}; }
};
template <typename T, int V> struct Source<T, V, true> {
    typedef SubCodes<V> Tokens;
    WaveRows rows, scales;
    uint32_t off, soff;
    template <int LR>
    __device__ __forceinline__ Source(const void*, const gdr2_rows8& p, int64_t row0, int64_t, int64_t C, const GlrLane<V, LR>& lane)
        : rows(WaveRows::at<uint8_t>(p.codes, row0, C)), scales(WaveRows::at<uint8_t>(p.scales, row0, scale_count(C))),
          off(lane.template offset<uint8_t>(rows.row_bytes)), soff(lane.scale_offset(scales.row_bytes, C))
    {
    }
    struct Reader {
        __amdgpu_buffer_rsrc_t codes, scales;
        RowOffset at, scale_at;
        __device__ __forceinline__ void load(int k, Tokens& to)
        {
            if constexpr (V == 2) {
                to.raw[k] = __builtin_amdgcn_raw_buffer_load_b16(codes, at.next(), 0, 0);
                // 16 lanes hold a block, as many as a sub-chunk has tokens; the last token's code is the last use
                static_assert(kRows8 / V == kGlrChunk, "one lane a token");
                if (k == kGlrChunk - 1)
                    to.scale[0] = __builtin_amdgcn_raw_buffer_load_b8(scales, scale_at.at + (threadIdx.x % kGlrChunk) * scale_at.row_bytes, 0, 0);
            } else {
                to.raw[k] = __builtin_amdgcn_raw_buffer_load_b8(codes, at.next(), 0, 0);
                to.scale[k] = __builtin_amdgcn_raw_buffer_load_b8(scales, scale_at.next(), 0, 0);
            }
        }
    };
    __device__ __forceinline__ Reader reader(int64_t first, int left) const
    {
        return {rows.buffer(first, left), scales.buffer(first, left), {off, rows.row_bytes}, {soff, scales.row_bytes}};
    }
};

// A sub-chunk's (P, L) through LDS: the gradient that reaches this lane's
// sub-chunk from behind, and in `lam` the one that leaves the tile.
template <int V, int LR, int N>
__device__ __forceinline__ void reverse_fold(const float (*s_span)[LR][2 * V], const GlrLane<V, LR>& lane, float (&lam)[V],
                                             float (&reach)[V])
{
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
        float pl[2 * V];
#pragma unroll
        for (int v = 0; v < 2 * V; ++v)
            pl[v] = s_span[j][lane.li][v];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            reach[v] = j == lane.sub || j == N - 1 ? lam[v] : reach[v];
            lam[v] = fmaf(pl[2 * v], lam[v], pl[2 * v + 1]);
        }
        if (j % 8 == 0)
            __builtin_amdgcn_sched_barrier(0);       // eight reads in flight at most
    }
}

template <int W> struct TileRows {
    int64_t n;
    int wave;
    __device__ __forceinline__ int64_t first(int64_t t) const { return t + wave * W; }
    __device__ __forceinline__ int left(int64_t t) const
    {
        const int64_t m = t < 0 ? 0 : n - first(t);
        return (int)(m < 0 ? 0 : m > W ? W : m);
    }
    // the wave's first token, where it has one
    __device__ __forceinline__ int64_t at(int64_t t) const { return left(t) > 0 ? first(t) : 0; }
};

template <bool CHAINED> constexpr int kWaves = CHAINED ? kChainedBackwardWaves : kGlrWaves;

template <typename T, int V, int LR, bool P8, bool CHAINED>
__global__ __launch_bounds__(64 * kWaves<CHAINED>, CHAINED ? 3 : 2) void glr_backward_kernel(gdr2_glr_bwd_args p, GlrPlan plan, GlrChain chain, float* part)
{
    typedef GlrTile<LR, kWaves<CHAINED>> Tile;
    __shared__ float s_span[CHAINED ? 1 : 2][Tile::kSubs][LR][2 * V];
    __shared__ float s_state[CHAINED ? LR * V : 1];
    const gdr2_glr_args& a = p.f;
    const GlrWork work = CHAINED ? chained_work(plan, chain, true) : one_pass_work(plan);
    const Segment seg = segment_of(plan, work.slot);
    const GlrLane<V, LR> lane(a.C, work.block);
    const int64_t c64 = work.block * (LR * V) + threadIdx.x;       // the first wave's channels, one a lane
    if (CHAINED && seg.q.seq < 0)
        chain_idle(chain, work.slot, a.C, c64);
    float dA[V], A2[V], Av[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Av[v] = lane.on ? finite(a.A[lane.c + v]) : 0.f;
        A2[v] = exponent_scale(Av[v]);
        dA[v] = 0.f;
    }
    if (seg.q.seq >= 0) {
        const int64_t row0 = seg.q.row0 + seg.t0;
        const TileRows<Tile::kWaveTokens> rows{seg.n, lane.wave};
        const Source<T, V, P8> sx(a.x, a.x8, row0, a.x_stride, a.C, lane), sr(a.r, a.r8, row0, a.r_stride, a.C, lane),
            si(a.i, a.i8, row0, a.i_stride, a.C, lane);
        const Source<T, V, false> sd(p.dy, row0, a.C, lane);
        const WaveRows ox = WaveRows::at<T>(p.dx, row0, a.C), orr = WaveRows::at<T>(p.dr, row0, a.C), oi = WaveRows::at<T>(p.di, row0, a.C);
        const uint32_t off = lane.template offset<T>(ox.row_bytes);
        const int64_t chunk0 = chunk_row(a, seg.q) + seg.t0 / kGlrChunk;
        // tiles behind this one
        const int64_t L = (int64_t)1 << plan.seg.lg, count = (seg.q.len + L - 1) >> plan.seg.lg, behind = count > 0 ? count - 1 - seg.q.index : 0;
        float lam[V], reach[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            lam[v] = 0.f;
        if (!CHAINED && p.dh_out && lane.on)
            load_channels<V>(p.dh_out + seg.q.seq * a.C + lane.c, lam);

        // the next tile's tokens take the registers of this one's as these are used up: every load runs most of a
        // tile ahead of its use, and they go out evenly over the tile
        typename Source<T, V, P8>::Tokens x, r, i;
        SubRows<T, V> dy;
        float h0[V];
        auto load_state = [&](int64_t t) {
            const int mine = rows.left(t) - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
#pragma unroll
            for (int v = 0; v < V; ++v)
                h0[v] = 0.f;
            if (lane.on && mine > 0)
                load_channels<V>(a.h_chunks + (chunk0 + t / kGlrChunk + lane.sub) * a.C + lane.c, h0);
        };
        // a tile of an empty sequence hands on what it is handed
        const int64_t last = seg.n > 0 ? (seg.n - 1) / Tile::kTokens * Tile::kTokens : CHAINED ? 0 : -1;
        if (last >= 0) {
            const int m = rows.left(last);
            const int64_t first = rows.at(last);
            auto nr = sr.reader(first, m), nx = sx.reader(first, m), ni = si.reader(first, m);
            auto nd = sd.reader(first, m);
#pragma unroll
            for (int k = 0; k < kGlrChunk; ++k) {
                nr.load(k, r);
                nd.load(k, dy);
            }
#pragma unroll
            for (int k = 0; k < kGlrChunk; ++k) {
                nx.load(k, x);
                ni.load(k, i);
            }
            load_state(last);
        }
        int buf = 0;
        for (int64_t t = last; CHAINED || t >= 0; t -= Tile::kTokens) {
            const int left = rows.left(t), mine = left - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
            const int64_t ahead = t - Tile::kTokens;
            const int nleft = rows.left(ahead);
            auto nr = sr.reader(rows.at(ahead), nleft), nx = sx.reader(rows.at(ahead), nleft), ni = si.reader(rows.at(ahead), nleft);
            auto nd = sd.reader(rows.at(ahead), nleft);
            // Chained, only the gate s(r) is kept from here to the gradients' recurrence, not a: the exponential is
            // evaluated again there, which costs less than the registers (three waves a SIMD instead of two).
            float sg[kGlrChunk][V], at[kGlrChunk][V], g[kGlrChunk][V], P[V], Lr[V];
            tokens_up([&](auto at_k) {
                constexpr int K = decltype(at_k)::value;
                float rv[V];
                token_of<K>(r, rv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    sg[K][v] = kept_gate(rv[v]);
                    here(sg[K][v]);
                }
            });
            // (loads stay behind the uses of what was in their registers)
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!CHAINED) {
#pragma unroll
                for (int k = 0; k < kGlrChunk; ++k)
                    nr.load(k, r);
            }
            __builtin_amdgcn_sched_barrier(0);
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
                    const float e = fast_exp2(A2[v] * gate_of(sg[k][v]));
                    Lr[v] = e * (dy.get(k, v) + Lr[v]);
                    P[v] *= e;
                    // the gate's value is formed again where it is used (one pass has the registers to hold half of them)
                    if (CHAINED || k >= kGlrChunk / 2)
                        here(sg[k][v]);
                    if constexpr (!CHAINED)
                        at[k][v] = e;
                }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s_span[buf][lane.sub][lane.li][2 * v] = P[v];
                s_span[buf][lane.sub][lane.li][2 * v + 1] = Lr[v];
            }
            lds_barrier();
            if constexpr (CHAINED) {
                if (lane.wave == 0)
                    s_state[threadIdx.x] = chain_state<V, LR, Tile::kSubs, -1>(chain, s_span[0], work.slot, behind, a.C, c64,
                                                                  p.dh_out ? p.dh_out + seg.q.seq * a.C : nullptr);
                lds_barrier();
#pragma unroll
                for (int v = 0; v < V; ++v)
                    lam[v] = s_state[lane.li * V + v];
            }
            reverse_fold<V, LR, Tile::kSubs>(s_span[buf], lane, lam, reach);
            float h[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = h0[v];
#pragma unroll
            for (int k = kGlrChunk - 1; k >= 0; --k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if constexpr (CHAINED)
                        at[k][v] = fast_exp2(A2[v] * gate_of(sg[k][v]));
                    g[k][v] = dy.get(k, v) + reach[v];
                    reach[v] = at[k][v] * g[k][v];
                    here(g[k][v]);
                    if constexpr (CHAINED)
                        here(sg[k][v]);
                }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!CHAINED) {
#pragma unroll
                for (int k = 0; k < kGlrChunk; ++k)
                    nd.load(k, dy);
                load_state(ahead);
            }
            __builtin_amdgcn_sched_barrier(0);
            const int64_t first = rows.at(t);
            const auto bx = ox.buffer(first, left), br = orr.buffer(first, left), bi = oi.buffer(first, left);
            RowOffset to{off, ox.row_bytes};
            tokens_up([&](auto at_k) {
                constexpr int K = decltype(at_k)::value;
                float xv[V], iv[V], dx[V], dr[V], di[V];
                token_of<K>(x, xv);
                token_of<K>(i, iv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float s = gate_of(sg[K][v]), e = at[K][v], q = glr_root(A2[v] * s, e);
                    // a masked token's x and i have no part, whatever they hold
                    const float ei = fast_exp2(-kLog2e * iv[v]), all = __builtin_amdgcn_rcpf(1.f + ei);
                    const float o = unless_masked(q, all), in = unless_masked(q, all * xv[v]);
                    const float gq = g[K][v] * q;
                    dx[v] = gq * o;
                    // s(i) (1 - s(i)) as s(i)^2 e^-i: the difference would cancel where the gate is open.  (Where the
                    // exponential is infinite, or i a masked NaN, `in` is 0.)
                    di[v] = in * fminf(ei, __FLT_MAX__) * dx[v];
                    // a/q where q is 0: anything finite, for `in` is 0
                    const float over = e * __builtin_amdgcn_rcpf(fmaxf(q, 1e-30f));
                    const float du = g[K][v] * e * fmaf(-in, over, h[v]);
                    dA[v] = fmaf(du, s, dA[v]);
                    dr[v] = du * (Av[v] * gate_slope(sg[K][v]));
                    h[v] = fmaf(e, h[v], q * in);
                }
                const uint32_t place = to.next();
                store_token<T, V>(bx, place, dx);
                store_token<T, V>(br, place, dr);
                store_token<T, V>(bi, place, di);
                // tokens are scheduled four at a time: more of them in flight would not fit the registers
                if constexpr (K % 4 == 3) {
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (!CHAINED) {
#pragma unroll
                        for (int k = K - 3; k <= K; ++k) {
                            nx.load(k, x);
                            ni.load(k, i);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            });
            if constexpr (CHAINED)
                break;
            buf ^= 1;
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
        store_channels<V>(part + work.slot * a.C + lane.c, dA);
    }
}

template <typename T, int V, int LR, bool P8> hipError_t backward_lr(const gdr2_glr_bwd_args& p, hipStream_t stream)
{
    const GlrPlan plan = glr_plan(p.f, V, true);
    const dim3 grid((unsigned)(plan.seg.slots() * plan.blocks)), threads(64 * (plan.chained ? kWaves<true> : kWaves<false>));
    float* part = (float*)((uint64_t*)p.workspace + plan.chain_words());
    const int64_t P = p.f.B > 0 ? plan.seg.slots() : 0;
    if (P > 0) {
        if (plan.chained) {
            const hipError_t e = launch_glr_chain_reset(plan, p.workspace, stream);
            if (e != hipSuccess)
                return e;
            hipLaunchKernelGGL((glr_backward_kernel<T, V, LR, P8, true>), grid, threads, 0, stream, p, plan, plan.chain(p.workspace), part);
        } else {
            hipLaunchKernelGGL((glr_backward_kernel<T, V, LR, P8, false>), grid, threads, 0, stream, p, plan, GlrChain{}, part);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return launch_column_sum(part, P, p.f.C, {p.dA, p.f.C}, {nullptr, 0}, {nullptr, 0}, stream);
}

template <bool P8> hipError_t backward_p(const gdr2_glr_bwd_args& p, hipStream_t stream)
{
    if (glr_pairs(p.f))
        return backward_lr<bf16, 2, 32, P8>(p, stream);
    return p.f.dtype == GDR2_BF16 ? backward_lr<bf16, 1, 64, P8>(p, stream) : backward_lr<float, 1, 64, P8>(p, stream);
}

}  // namespace

// The largest of the needs that the pointers decide between.
size_t glr_backward_workspace_bytes(const gdr2_glr_bwd_args& p)
{
    int64_t most = 0;
    for (int V : {1, 2})
        for (const void* x : {(const void*)nullptr, (const void*)&p}) {       // none or any
            gdr2_glr_args f = p.f;
            f.x = x;
            const GlrPlan plan = glr_plan(f, V, true);
            most = std::max(most, plan.chain_words() * 8 + plan.seg.slots() * p.f.C * 4);
        }
    return p.f.B > 0 ? (size_t)most : 0;
}

hipError_t launch_glr_backward(const gdr2_glr_bwd_args& p, hipStream_t stream)
{
    return p.f.x ? backward_p<false>(p, stream) : backward_p<true>(p, stream);
}

int64_t glr_launch_groups(const gdr2_glr_args& a, bool backward)
{
    int64_t most = 0;
    for (int V : {1, 2}) {
        const GlrPlan plan = glr_plan(a, V, backward);
        const int waves = plan.chained && backward ? kChainedBackwardWaves : kGlrWaves;
        const double groups = (double)plan.seg.slots() * (double)plan.blocks * (waves * 64 / 256);
        most = groups >= (double)kMaxGroups ? kMaxGroups : std::max(most, (int64_t)groups);
    }
    return most;
}

}  // namespace gdr2
