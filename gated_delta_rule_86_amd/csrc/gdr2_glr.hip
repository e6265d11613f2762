// gdr2_glr.hip -- gated linear recurrence, forwards and one token at a time.
//
//   a_t = exp(A s(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t,  y_t = h_t
//
// 8 bytes an element of bf16 rows, and about 45 vector operations, six of them
// transcendental (a quarter of the rate): both near what the chip does in the same time.
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

// (a, b) of a sub-chunk, and its (P, L).
template <typename T, int V>
__device__ __forceinline__ SpanVec<V> form_terms(const Inputs<T, V>& in, const float (&A2)[V], float (&a)[kGlrChunk][V],
                                                 float (&b)[kGlrChunk][V])
{
    SpanVec<V> s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        s.p[v] = 1.f;
        s.l[v] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kGlrChunk; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float sr = sigmoid_f(in.r.get(k, v)), si = sigmoid_f(in.i.get(k, v));
            const float at = glr_decay(A2[v], sr), q = glr_root(A2[v], sr, at);
            a[k][v] = at;
            // a masked token's input may be anything, NaN among it
            b[k][v] = q == 0.f ? 0.f : q * si * in.x.get(k, v);
            s.l[v] = fmaf(at, s.l[v], b[k][v]);
            s.p[v] *= at;
        }
    return s;
}

// What a workgroup needs to walk the tiles of its segment.
template <typename T, int V, int LR> struct Walk {
    typedef GlrTile<LR> Tile;
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
    __device__ __forceinline__ int64_t first(int64_t t) const { return t + wave * Tile::kWaveTokens; }
    __device__ __forceinline__ int left(int64_t t) const
    {
        const int64_t m = n - first(t);
        return (int)(m < 0 ? 0 : m > Tile::kWaveTokens ? Tile::kWaveTokens : m);
    }
    __device__ __forceinline__ void load(Inputs<T, V>& in, int64_t t) const
    {
        const int m = left(t);
        // no row past the segment is addressed, not even by a descriptor without bytes
        const int64_t at = m > 0 ? first(t) : 0;
        in.r.load(r.buffer(at, m), orr, r.row_bytes);
        in.x.load(x.buffer(at, m), ox, x.row_bytes);
        in.i.load(i.buffer(at, m), oi, i.row_bytes);
    }
};

// The rows of one array of a sub-chunk in 8 bits.
template <typename T, int V, int LR>
__device__ __forceinline__ void put_codes(const gdr2_rows8& to, const SubRows<T, V>& rows, int64_t C, int64_t row, int left,
                                          const GlrLane<V, LR>& lane)
{
    constexpr int LPB = kRows8 / V;
    const int64_t nb = scale_count(C);
#pragma unroll
    for (int k = 0; k < kGlrChunk; ++k) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = rows.get(k, j);
        const int amax = block_max<V>(v, lane.on), e = block_exponent(amax);
        Codes<V> codes;
        codes.pack(v, amax, e);
        if (lane.on && k < left) {
            codes.store((uint8_t*)to.codes + (row + k) * C + lane.c);
            if (lane.li % LPB == 0)
                ((uint8_t*)to.scales)[(row + k) * nb + lane.c / kRows8] = (uint8_t)(e + 127);
        }
    }
}

// The state the segment starts from: h0 and the segments before it in turn,
// eight of their (P, L) in flight.
template <int V>
__device__ __forceinline__ void start_state(const float* h0, const float* spans, const Piece& q, int64_t C, int64_t c, bool on,
                                            float (&h)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        h[v] = 0.f;
    if (!on)
        return;
    if (h0)
        load_channels<V>(h0 + q.seq * C + c, h);
    const float* s = spans + (q.first * C + c) * 2;
    for (int64_t j = 0; j < q.index; j += kFoldAhead) {
        float pl[kFoldAhead][2 * V];
#pragma unroll
        for (int u = 0; u < kFoldAhead; ++u)
            if (j + u < q.index)
                load_channels<2 * V>(s + (j + u) * C * 2, pl[u]);
#pragma unroll
        for (int u = 0; u < kFoldAhead; ++u)
            if (j + u < q.index)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    h[v] = fmaf(pl[u][2 * v], h[v], pl[u][2 * v + 1]);
    }
}

// SPAN: (P, L) of every segment but a sequence's last one, nothing else.
template <typename T, int V, int LR, bool PACK, bool SPAN>
__global__ __launch_bounds__(64 * kGlrWaves) void glr_forward_kernel(gdr2_glr_args a, GlrPlan plan, float* spans)
{
    typedef GlrTile<LR> Tile;
    __shared__ float s_span[2][Tile::kSubs][LR][2 * V];
    const int64_t slot = blockIdx.x / plan.blocks, block = blockIdx.x - slot * plan.blocks;
    const Segment seg = segment_of(plan, slot);
    if (seg.q.seq < 0 || (SPAN && seg.t0 + seg.n >= seg.q.len))
        return;
    const GlrLane<V, LR> lane(a.C, block);
    const int64_t row0 = seg.q.row0 + seg.t0;
    const Walk<T, V, LR> walk(a, row0, seg.n, lane);
    float A2[V], h[V], whole[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A2[v] = lane.on ? exponent_scale(a.A[lane.c + v]) : 0.f;
        h[v] = 0.f;
        whole[v] = 1.f;
    }
    if constexpr (!SPAN)
        start_state<V>(a.h0, spans, seg.q, a.C, lane.c, lane.on, h);
    const WaveRows y = WaveRows::at<T>(a.y, row0, a.C);
    const uint32_t oy = lane.template offset<T>(y.row_bytes);
    const int64_t chunk0 = a.h_chunks ? chunk_row(a, seg.q) + seg.t0 / kGlrChunk : 0;

    Inputs<T, V> next;
    walk.load(next, 0);
    int buf = 0;
    for (int64_t t = 0; t < seg.n; t += Tile::kTokens, buf ^= 1) {
        Inputs<T, V> cur = next;
        walk.load(next, t + Tile::kTokens);
        const int left = walk.left(t), mine = left - (lane.sub - lane.wave * Tile::kGroups) * kGlrChunk;
        const int64_t first = t + lane.sub * kGlrChunk;       // of this sub-chunk in the segment
        if constexpr (PACK) {
            put_codes<T, V, LR>(a.x8, cur.x, a.C, row0 + first, mine, lane);
            put_codes<T, V, LR>(a.r8, cur.r, a.C, row0 + first, mine, lane);
            put_codes<T, V, LR>(a.i8, cur.i, a.C, row0 + first, mine, lane);
        }
        if (left < Tile::kWaveTokens)
            cur.r.mask(mine);
        float at[kGlrChunk][V], b[kGlrChunk][V];
        const SpanVec<V> s = form_terms<T, V>(cur, A2, at, b);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s_span[buf][lane.sub][lane.li][2 * v] = s.p[v];
            s_span[buf][lane.sub][lane.li][2 * v + 1] = s.l[v];
        }
        // one barrier a tile: a buffer is written again two tiles on, when every wave has passed
        // the barrier between, and so read it
        lds_barrier();
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
                if constexpr (SPAN)
                    whole[v] *= pl[2 * v];
            }
        }
        if constexpr (!SPAN) {
            if (a.h_chunks && lane.on && mine > 0)
                store_channels<V>(a.h_chunks + (chunk0 + first / kGlrChunk) * a.C + lane.c, start);
            const auto out = y.buffer(left > 0 ? walk.first(t) : 0, left);
#pragma unroll
            for (int k = 0; k < kGlrChunk; ++k) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    start[v] = fmaf(at[k][v], start[v], b[k][v]);
                store_token<T, V>(out, oy + k * y.row_bytes, start);
            }
        }
    }
    if (lane.sub != 0 || !lane.on)
        return;
    if constexpr (SPAN) {
        float* to = spans + (slot * a.C + lane.c) * 2;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            to[2 * v] = whole[v];
            to[2 * v + 1] = h[v];
        }
    } else if (a.h_out && seg.t0 + seg.n == seg.q.len) {
        store_channels<V>(a.h_out + seg.q.seq * a.C + lane.c, h);
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
            const float at_ = glr_decay(A2, sr), q = glr_root(A2, sr, at_);
            h[v] = fmaf(at_, h[v], q == 0.f ? 0.f : q * si * x[v]);
        }
        store_row<V>(a.state + n * a.C + c, h);
        store_row<V>((T*)a.y + n * a.C + c, h);
    }
}

int64_t span_floats(const gdr2_glr_args& a, const GlrPlan& p) { return p.split ? p.seg.slots() * a.C * 2 : 0; }

template <typename T, int V, int LR> hipError_t forward_lr(const gdr2_glr_args& a, const GlrPlan& plan, hipStream_t stream)
{
    const dim3 grid((unsigned)(plan.seg.slots() * plan.blocks)), threads(64 * kGlrWaves);
    float* spans = (float*)a.workspace;
    if (plan.split) {
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, false, true>), grid, threads, 0, stream, a, plan, spans);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (a.x8.codes)
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, true, false>), grid, threads, 0, stream, a, plan, spans);
    else
        hipLaunchKernelGGL((glr_forward_kernel<T, V, LR, false, false>), grid, threads, 0, stream, a, plan, spans);
    return hipGetLastError();
}

template <typename T> hipError_t forward_t(const gdr2_glr_args& a, hipStream_t stream)
{
    if (!glr_pairs(a))
        return forward_lr<T, 1, 64>(a, glr_plan(a, 1, false), stream);
    const GlrPlan plan = glr_plan(a, 2, false);
    return plan.lr == 32 ? forward_lr<T, 2, 32>(a, plan, stream) : forward_lr<T, 2, 16>(a, plan, stream);
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

// One workgroup walks a sequence when that gives at least three workgroups for
// four compute units, with half as many channels each where that makes the
// difference.  Otherwise sequences are cut into segments, for two workgroups a
// compute unit.
GlrPlan glr_plan(const gdr2_glr_args& a, int V, bool backward)
{
    GlrPlan p{{a.offsets, a.B, a.T, 40}, 0, V == 2 ? 32 : 64, false};
    const int64_t units = device_cu_count(), B = std::max(a.B, (int64_t)1);
    auto blocks = [&](int lr) { return ceil_div(a.C, (int64_t)lr * V); };
    auto enough = [&](int lr) { return B * blocks(lr) * 4 >= units * 3; };
    bool split = a.algo == GDR2_ALGO_SEGMENTED;
    if (a.algo != GDR2_ALGO_SEGMENTED && !enough(p.lr)) {
        if (V == 2)
            p.lr = 16;
        split = a.algo == GDR2_ALGO_AUTO && !enough(p.lr);
        if (split && V == 2)
            p.lr = 32;
    }
    p.blocks = blocks(p.lr);
    if (split) {
        // a dense sequence has T tokens; a packed one has T / B on average
        const int64_t tokens = a.offsets ? a.T : B * a.T, want = ceil_div(units * 2, p.blocks);
        int lg = a.algo == GDR2_ALGO_SEGMENTED ? 7 : 9;
        while (lg < 40 && (tokens >> lg) > want)
            ++lg;
        p.split = a.offsets ? (a.T >> lg) > 0 : a.T > ((int64_t)1 << lg);
        if (p.split)
            p.seg.lg = lg;
    }
    return p;
}

// The larger of the two widths' needs where the pointers decide between them.
size_t glr_workspace_bytes(const gdr2_glr_args& a)
{
    const int64_t one = span_floats(a, glr_plan(a, 1, false)), two = a.C % 2 ? 0 : span_floats(a, glr_plan(a, 2, false));
    return (size_t)std::max(one, two) * sizeof(float);
}

hipError_t launch_glr_forward(const gdr2_glr_args& a, hipStream_t stream)
{
    return a.dtype == GDR2_BF16 ? forward_t<bf16>(a, stream) : forward_t<float>(a, stream);
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
