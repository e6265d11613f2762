// gdr2_glr.hip -- gated linear recurrence, forwards and one token at a time.
//
//   a_t = exp(A s(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t,  y_t = h_t
//
// 8 bytes an element of bf16 rows, and 34 vector operations, six of them
// transcendental: memory bounds it, with the vector units busy for 60 % of
// the time.  8x4096x2048 in 112 us (4.8 TB/s; a large copy 5.15), one sequence of
// 32768 tokens, in chained tiles, 124 and 5 for emptying the chain.  Writing
// the inputs in 8 bits makes that 11.3 bytes and 57 operations: 4x4096x2048
// 99 us (3.8 TB/s), both at half of what they could be by themselves, because a
// tile loads, computes and stores in turn and 116 registers leave four waves a SIMD.
// (The one-pass variant of two channels a lane holds 128 registers and two spilled ones.)
// gdr2_glr.h describes the layout.
#include <algorithm>

#include "gdr2_glr.h"

namespace gdr2 {

namespace {

template <int V> struct SpanVec {
    float p[V], l[V];
};

// The inputs of one tile's sub-chunk.
template <typename T, int V> struct Inputs {
    SubRows<T, V> x, r, i;
};

// The rows of x, r and i, from the segment's first one on.
template <typename T, int V, int LR> struct Walk {
    static constexpr int kWaveTokens = 64 / LR * kGlrChunk;
    WaveRows x, r, i;
    uint32_t ox, orr, oi;
    int64_t n;          // tokens of the segment
    int wave;

    __device__ __forceinline__ Walk(const gdr2_glr_args& a, int64_t row0, int64_t n_, const GlrLane<V, LR>& lane)
        : x(WaveRows::at<T>(a.x, row0, a.x_stride)), r(WaveRows::at<T>(a.r, row0, a.r_stride)),
          i(WaveRows::at<T>(a.i, row0, a.i_stride)), ox(lane.template offset<T>(x.row_bytes)),
          orr(lane.template offset<T>(r.row_bytes)), oi(lane.template offset<T>(i.row_bytes)), n(n_), wave(lane.wave)
    {
    }
    // first token of this wave in the tile at `t`, and how many of its tokens exist
    __device__ __forceinline__ int64_t first(int64_t t) const { return t + wave * kWaveTokens; }
    __device__ __forceinline__ int left(int64_t t) const
    {
        const int64_t m = n - first(t);
        return (int)(m < 0 ? 0 : m > kWaveTokens ? kWaveTokens : m);
    }
    // f(buffers of r, x and i, offsets) of the tile at t
    template <typename F> __device__ __forceinline__ void with_tile(int64_t t, const F& f) const
    {
        const int m = left(t);
        // no row past the segment is addressed, not even by a descriptor without bytes
        const int64_t at = m > 0 ? first(t) : 0;
        f(r.buffer(at, m), x.buffer(at, m), i.buffer(at, m), RowOffset{orr, r.row_bytes}, RowOffset{ox, x.row_bytes},
          RowOffset{oi, i.row_bytes});
    }
};

// (a, b) of a sub-chunk, and its (P, L).  AHEAD: the registers of r and i are
// loaded again, for the tile at `t`, as soon as a token's terms are formed: the loads run a
// tile ahead of their use, and go out evenly over the tile.
template <bool AHEAD, int POLICY, typename T, int V, int LR>
__device__ __forceinline__ SpanVec<V> form_terms(Inputs<T, V>& in, const Walk<T, V, LR>& walk, int64_t t, const float (&A2)[V],
                                                 float (&a)[kGlrChunk][V], float (&b)[kGlrChunk][V])
{
    SpanVec<V> s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s.p[v] = 1.f;
        s.l[v] = 0.f;
    }
    walk.with_tile(t, [&](auto br, auto bx, auto bi, RowOffset atr, RowOffset atx, RowOffset ati) {
#pragma unroll
        for (int k = 0; k < kGlrChunk; ++k) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float sr = sigmoid_f(in.r.get(k, v)), si = sigmoid_f(in.i.get(k, v));
                const float u = A2[v] * sr, at = fast_exp2(u), q = glr_root(u, at);
                a[k][v] = at;
                b[k][v] = unless_masked(q, q * si * in.x.get(k, v));
                here(b[k][v]);
                s.l[v] = fmaf(at, s.l[v], b[k][v]);
                s.p[v] *= at;
            }
            if constexpr (AHEAD) {
                in.r.template load<POLICY>(k, br, atr);
                in.i.template load<POLICY>(k, bi, ati);
            }
        }
    });
    return s;
}

// ---- rows in 8 bits --------------------------------------------------------
// The largest magnitudes of the 16 tokens over the 16 lanes of a block, lane k
// of the block returning that of token k: each round hands half of the tokens to
// the partner that keeps them.  Magnitudes are pairs of 16-bit integers that
// order like the bf16 numbers they are the bits of.
__device__ __forceinline__ int pair_max(int a, int b)
{
    return __builtin_bit_cast(int, __builtin_elementwise_max(__builtin_bit_cast(s16x2, a), __builtin_bit_cast(s16x2, b)));
}
template <int CTRL, int N> __device__ __forceinline__ void max_round(int (&m)[N], bool upper)
{
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const int keep = upper ? m[k + N / 2] : m[k], give = upper ? m[k] : m[k + N / 2];
        m[k] = pair_max(keep, __builtin_amdgcn_update_dpp(0, give, CTRL, 0xF, 0xF, true));
    }
}
__device__ __forceinline__ int token_max(const int (&in)[16])
{
    const int lane = threadIdx.x;
    int m[16], n[8], o[4], p[2];
#pragma unroll
    for (int k = 0; k < 16; ++k)
        m[k] = in[k];
    max_round<0x140>(m, lane & 8);       // lane 15 - i
#pragma unroll
    for (int k = 0; k < 8; ++k)
        n[k] = m[k];
    max_round<0x141>(n, lane & 4);       // lane 7 - i of the eight
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = n[k];
    max_round<0x4E>(o, lane & 2);        // lane i ^ 2
    p[0] = o[0];
    p[1] = o[1];
    max_round<0xB1>(p, lane & 1);        // lane i ^ 1
    const s16x2 v = __builtin_bit_cast(s16x2, p[0]);
    return v[0] > v[1] ? v[0] : v[1];
}

// The rows of one array of a sub-chunk in 8 bits.
template <typename T, int V> struct CodeRows {
    WaveRows codes, scales;
    uint32_t off, soff;
    template <int LR> __device__ __forceinline__ CodeRows(const gdr2_rows8& to, int64_t row0, int64_t C, const GlrLane<V, LR>& lane)
        : codes(WaveRows::at<uint8_t>(to.codes, row0, C)), scales(WaveRows::at<uint8_t>(to.scales, row0, scale_count(C))),
          off(lane.template offset<uint8_t>(codes.row_bytes)), soff(lane.scale_offset(scales.row_bytes, C))
    {
    }
    __device__ __forceinline__ void put(const SubRows<T, V>& rows, bool on, int64_t first, int left) const
    {
        const auto bc = codes.buffer(first, left), bs = scales.buffer(first, left);
        RowOffset at{off, codes.row_bytes};
        const s16x2 none = {0, 0};
        if constexpr (V == 2) {
            // |v| + 0x80 is negative as a 16-bit integer for NaN and infinities, and above 0 otherwise
            int m[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
                m[k] = on ? __builtin_bit_cast(int, __builtin_bit_cast(s16x2, rows.raw[k] & 0x7fff7fffu) + (s16x2){0x80, 0x80}) : 0;
            const int most = token_max(m);
            const int e = block_exponent(most > 0 ? (most - 0x80) << 16 : -1);
            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(e + 127), bs, soff + (threadIdx.x % 16) * scales.row_bytes, 0, 0);
            const int scale = (e + 127) << 23;
            uint32_t c[16];
            // asked for every block of the row: a lane's token is another's than its channels, so that in the
            // last block lanes past the row's end have tokens too
            if (__any(most <= 0 && soff < kNowhere))
                codes_of<true, 0>(rows, scale, most > 0, c);
            else
                codes_of<false, 0>(rows, scale, true, c);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)c[k], bc, at.next(), 0, 0);
        } else {
            RowOffset sat{soff, scales.row_bytes};
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float v[1] = {rows.get(k, 0)};
                const int amax = block_max<1>(v, on ? 1 : 0), e = block_exponent(amax);
                const float clipped = amax < 0 ? clip_infinity(v[0]) : v[0];
                const s16x2 c = codes2<false>(clipped, 0.f, amax < 0 ? 1.f : scale_of(e + 127), none);
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)c[0], bc, at.next(), 0, 0);
                const uint32_t place = sat.next();
                if (threadIdx.x % kRows8 == 0)
                    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(e + 127), bs, place, 0, 0);
            }
        }
    }
    // Token K's scale lies in lane K of the block.  ODD: some block of the wave is without numbers.
    template <bool ODD, int K>
    __device__ __forceinline__ void codes_of(const SubRows<T, V>& rows, int scale, bool number, uint32_t (&out)[16]) const
    {
        if constexpr (K < 16) {
            typedef __bf16 Pair __attribute__((ext_vector_type(2)));
            const s16x2 none = {0, 0};
            const float s = __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, scale, 0x150 + K, 0xF, 0xF, true));
            s16x2 c = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(none, __builtin_bit_cast(Pair, rows.raw[K]), s, false);
            if constexpr (ODD) {
                const bool some = __builtin_amdgcn_update_dpp(0, (int)number, 0x150 + K, 0xF, 0xF, true);
                const s16x2 clipped = codes2<false>(clip_infinity(rows.get(K, 0)), clip_infinity(rows.get(K, 1)), 1.f, none);
                c = some ? c : clipped;
            }
            out[K] = __builtin_bit_cast(uint32_t, c);
            codes_of<ODD, K + 1>(rows, scale, number, out);
        }
    }
};

template <typename T, int V, int LR, int POLICY, bool PACK, bool CHAINED>
__global__ __launch_bounds__(64 * kGlrWaves, PACK ? 2 : 4) void glr_forward_kernel(gdr2_glr_args a, GlrPlan plan, GlrChain chain)
{
    typedef GlrTile<LR, kGlrWaves> Tile;
    __shared__ float s_span[CHAINED ? 1 : 2][Tile::kSubs][LR][2 * V];
    __shared__ float s_state[CHAINED ? LR * V : 1];
    const GlrWork work = CHAINED ? chained_work(plan, chain, false) : one_pass_work(plan);
    const Segment seg = segment_of(plan, work.slot);
    const int64_t c64 = work.block * (LR * V) + threadIdx.x;       // the first wave's channels, one a lane
    if (seg.q.seq < 0) {
        if constexpr (CHAINED)
            chain_idle(chain, work.slot, a.C, c64);
        return;
    }
    const GlrLane<V, LR> lane(a.C, work.block);
    const int64_t row0 = seg.q.row0 + seg.t0;
    const Walk<T, V, LR> walk(a, row0, seg.n, lane);
    float A2[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A2[v] = lane.on ? exponent_scale(a.A[lane.c + v]) : 0.f;
        h[v] = 0.f;
    }
    if (!CHAINED && a.h0 && lane.on)
        load_channels<V>(a.h0 + seg.q.seq * a.C + lane.c, h);
    const WaveRows y = WaveRows::at<T>(a.y, row0, a.C);
    const uint32_t oy = lane.template offset<T>(y.row_bytes);
    const int64_t chunk0 = a.h_chunks ? chunk_row(a, seg.q) + seg.t0 / kGlrChunk : 0;
    const CodeRows<T, V> x8(a.x8, row0, a.C, lane), r8(a.r8, row0, a.C, lane), i8(a.i8, row0, a.C, lane);

    Inputs<T, V> in;
    walk.with_tile(0, [&](auto br, auto bx, auto bi, RowOffset atr, RowOffset atx, RowOffset ati) {
#pragma unroll
        for (int k = 0; k < kGlrChunk; ++k) {
            in.r.template load<POLICY>(k, br, atr);
            in.x.template load<POLICY>(k, bx, atx);
            in.i.template load<POLICY>(k, bi, ati);
        }
    });
    int buf = 0;
    // a tile of an empty sequence hands on what it is handed
    for (int64_t t = 0; CHAINED || t < seg.n; t += Tile::kTokens) {
        const int left = walk.left(t), mine = left - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
        if constexpr (PACK) {
            const int64_t at = left > 0 ? walk.first(t) : 0;
            x8.put(in.x, lane.on, at, left);
            __builtin_amdgcn_sched_barrier(0);       // one array after the other: their registers
            r8.put(in.r, lane.on, at, left);
            __builtin_amdgcn_sched_barrier(0);
            i8.put(in.i, lane.on, at, left);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (left < Tile::kWaveTokens)
            in.r.mask(mine);
        float at[kGlrChunk][V], b[kGlrChunk][V];
        const SpanVec<V> s = form_terms<!CHAINED, POLICY, T, V, LR>(in, walk, t + Tile::kTokens, A2, at, b);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_span[buf][lane.sub][lane.li][2 * v] = s.p[v];
            s_span[buf][lane.sub][lane.li][2 * v + 1] = s.l[v];
        }
        // one barrier a tile: a buffer is written again two tiles on, when every wave has passed
        // the barrier between, and so read it
        lds_barrier();
        if constexpr (CHAINED) {
            if (lane.wave == 0)
                s_state[threadIdx.x] = chain_state<V, LR, Tile::kSubs, 1>(chain, s_span[0], work.slot, seg.q.index, a.C, c64,
                                                             a.h0 ? a.h0 + seg.q.seq * a.C : nullptr);
            lds_barrier();
#pragma unroll
            for (int v = 0; v < V; ++v)
                h[v] = s_state[lane.li * V + v];
        }
        float start[V];
#pragma unroll
        for (int j = 0; j < Tile::kSubs; ++j) {
            float pl[2 * V];
#pragma unroll
            for (int v = 0; v < 2 * V; ++v)
                pl[v] = s_span[buf][j][lane.li][v];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                start[v] = j == lane.sub || j == 0 ? h[v] : start[v];
                h[v] = fmaf(pl[2 * v], h[v], pl[2 * v + 1]);
            }
            if (j % 4 == 3)
                __builtin_amdgcn_sched_barrier(0);
        }
        if (a.h_chunks && lane.on && mine > 0)
            store_channels<V>(a.h_chunks + (chunk0 + t / kGlrChunk + lane.sub) * a.C + lane.c, start);
        const auto out = y.buffer(left > 0 ? walk.first(t) : 0, left);
        RowOffset to{oy, y.row_bytes};
#pragma unroll
        for (int k = 0; k < kGlrChunk; ++k) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                start[v] = fmaf(at[k][v], start[v], b[k][v]);
            store_token<T, V>(out, to.next(), start);
        }
        if constexpr (!CHAINED) {
            walk.with_tile(t + Tile::kTokens, [&](auto, auto bx, auto, RowOffset, RowOffset atx, RowOffset) {
#pragma unroll
                for (int k = 0; k < kGlrChunk; ++k)
                    in.x.template load<POLICY>(k, bx, atx);
            });
            buf ^= 1;
        } else {
            break;
        }
    }
    if (a.h_out && lane.sub == 0 && lane.on && seg.t0 + seg.n == seg.q.len)
        store_channels<V>(a.h_out + seg.q.seq * a.C + lane.c, h);
}

__global__ __launch_bounds__(256) void glr_chain_reset_kernel(GlrChain chain, int64_t tickets, int64_t words)
{
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < words; at += step) {
        chain.maps[at] = kNoMap;
        chain.states[at] = 0;
        if (at < tickets)
            chain.tickets[at * kTicketWords] = 0;
    }
}

// One token of V adjacent channels a thread.
template <typename T, int V> __global__ __launch_bounds__(256) void glr_step_kernel(gdr2_glr_step_args a, int64_t per)
{
    const int64_t step = (int64_t)gridDim.x * 256, items = a.N * per;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < items; at += step) {
        const int64_t n = (at | per) >> 32 ? at / per : (int64_t)((uint32_t)at / (uint32_t)per), c = (at - n * per) * V;
        float x[V], r[V], i[V], h[V], A[V];
        Raw<T, V>::get(Raw<T, V>::load((const T*)a.x + n * a.x_stride + c), x);
        Raw<T, V>::get(Raw<T, V>::load((const T*)a.r + n * a.r_stride + c), r);
        Raw<T, V>::get(Raw<T, V>::load((const T*)a.i + n * a.i_stride + c), i);
        Raw<float, V>::get(Raw<float, V>::load(a.state + n * a.C + c), h);
        Raw<float, V>::get(Raw<float, V>::load(a.A + c), A);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float A2 = exponent_scale(A[v]), sr = sigmoid_f(r[v]), si = sigmoid_f(i[v]);
            const float u = A2 * sr, a_t = fast_exp2(u), q = glr_root(u, a_t);
            h[v] = fmaf(a_t, h[v], unless_masked(q, q * si * x[v]));
        }
        store_row<V>(a.state + n * a.C + c, h);
        store_row<V>((T*)a.y + n * a.C + c, h);
    }
}

template <typename T, int V, int LR, int POLICY> hipError_t forward_lr(const gdr2_glr_args& a, hipStream_t stream)
{
    const GlrPlan plan = glr_plan(a, V, false);
    const dim3 grid((unsigned)(plan.seg.slots() * plan.blocks)), threads(64 * kGlrWaves);
    GlrChain chain = {};
    if (plan.chained) {
        const hipError_t e = launch_glr_chain_reset(plan, a.workspace, stream);
        if (e != hipSuccess)
            return e;
        chain = plan.chain(a.workspace);
    }
    const bool pack = a.x8.codes;
    if (plan.chained && pack)
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, POLICY, true, true>), grid, threads, 0, stream, a, plan, chain);
    else if (plan.chained)
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, POLICY, false, true>), grid, threads, 0, stream, a, plan, chain);
    else if (pack)
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, POLICY, true, false>), grid, threads, 0, stream, a, plan, chain);
    else
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, POLICY, false, false>), grid, threads, 0, stream, a, plan, chain);
    return hipGetLastError();
}

template <typename T, int V> hipError_t step_v(const gdr2_glr_step_args& a, hipStream_t stream)
{
    const int64_t per = a.C / V, items = a.N * per;
    // one item a thread while that is at most 32 workgroups per compute unit, then they are walked
    const dim3 grid((unsigned)std::min(ceil_div(items, 256), (int64_t)device_cu_count() * 32));
    hipLaunchKernelGGL((glr_step_kernel<T, V>), grid, dim3(256), 0, stream, a, per);
    return hipGetLastError();
}

}  // namespace

// One workgroup walks a sequence where that fills the chip: workgroups in
// whole rounds of the compute units, or nearly (us, one pass and chained, bf16: forward
// 8x4096x2048 112 and 126, 4x4096x2048 93 and 72, 1x32768x2048 673 and 126).
// Otherwise tiles are chained, and so are packed sequences, whose lengths are
// not known here.
// Chained are also the two passes with many registers or much arithmetic, the
// gradients from rows as they are and the forward that writes rows in 8 bits,
// where arrays are larger than half of the last cache and blocks of channels
// are whole lines of wide rows: workgroups that start whenever another ends
// overlap better with memory than ones that go in step.  Gradients: 8x4096x2048
// 248 and 232, 4x4096x4096 235 and 210, 16x4096x1024 229 and 228, fp32
// 8x2048x2048 211 and 191; 8-bit rows: 221 and 203, 213 and 197, 215 and 202,
// 171 and 154.  On the other sides: 8x2048x2048 105 and 121, 32x4096x512 231
// and 246, 15x3001x1002 161 and 215; 93 and 103, 208 and 211, 140 and 202.
// (From rows in 8 bits one pass stays ahead: 8x4096x2048 192 and 234.)
GlrPlan glr_plan(const gdr2_glr_args& a, int V, bool backward)
{
    // a chained tile: 16 tokens of 32 or 64 lanes along the channels
    int lg = V == 2 ? 5 : 4;
    for (int waves = backward ? kChainedBackwardWaves : kGlrWaves; waves > 1; waves /= 2)
        ++lg;
    GlrPlan p{{a.offsets, a.B, a.T, 40}, ceil_div(a.C, (int64_t)64), false, a.C};
    const int64_t units = device_cu_count(), groups = std::max(a.B, (int64_t)1) * p.blocks, rounds = ceil_div(groups, units);
    const bool fills = groups * 4 >= rounds * units * 3;
    const int64_t row_bytes = a.C * (a.dtype == GDR2_BF16 ? 2 : 4);
    const bool heavy = (backward ? a.x != nullptr : a.x8.codes != nullptr) && a.C >= 1024 && row_bytes % 128 == 0 &&
                       (double)a.B * (double)a.T * (double)row_bytes >= 128.0 * (1 << 20);
    const bool wanted = a.algo == GDR2_ALGO_SEGMENTED || (a.algo == GDR2_ALGO_AUTO && (a.offsets || !fills || heavy));
    // (a packed sequence may have all of the rows)
    p.chained = wanted && a.T > ((int64_t)1 << lg);
    if (p.chained)
        p.seg.lg = lg;
    return p;
}

hipError_t launch_glr_chain_reset(const GlrPlan& plan, void* workspace, hipStream_t stream)
{
    const int64_t words = plan.seg.slots() * plan.C;
    const dim3 grid((unsigned)std::min(ceil_div(words, 256), (int64_t)device_cu_count() * 8));
    hipLaunchKernelGGL(glr_chain_reset_kernel, grid, dim3(256), 0, stream, plan.chain(workspace), plan.blocks, words);
    return hipGetLastError();
}

// The larger of the two widths' needs where the pointers decide between them.
size_t glr_workspace_bytes(const gdr2_glr_args& a)
{
    const int64_t one = glr_plan(a, 1, false).chain_words(), two = glr_plan(a, 2, false).chain_words();
    return a.B > 0 ? (size_t)std::max(one, two) * 8 : 0;
}

hipError_t launch_glr_forward(const gdr2_glr_args& a, hipStream_t stream)
{
    const bool lines = glr_whole_lines(a);
    if (glr_pairs(a))
        return lines ? forward_lr<bf16, 2, 32, kOnce>(a, stream) : forward_lr<bf16, 2, 32, kKeep>(a, stream);
    if (a.dtype == GDR2_BF16)
        return forward_lr<bf16, 1, 64, kKeep>(a, stream);      // rows at odd elements
    return lines ? forward_lr<float, 1, 64, kOnce>(a, stream) : forward_lr<float, 1, 64, kKeep>(a, stream);
}

hipError_t launch_glr_step(const gdr2_glr_step_args& a, hipStream_t stream)
{
    const bool bf = a.dtype == GDR2_BF16;
    const int64_t e = bf ? 2 : 4;
    const bool wide = rows_aligned(a.x, a.x_stride, a.C, e, 4) && rows_aligned(a.r, a.r_stride, a.C, e, 4) &&
                      rows_aligned(a.i, a.i_stride, a.C, e, 4);
    if (bf)
        return wide ? step_v<bf16, 4>(a, stream) : step_v<bf16, 1>(a, stream);
    return wide ? step_v<float, 4>(a, stream) : step_v<float, 1>(a, stream);
}

}  // namespace gdr2
