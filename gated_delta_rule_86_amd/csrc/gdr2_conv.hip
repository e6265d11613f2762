// gdr2_conv.hip -- the short causal depthwise convolution: prompts, single
// tokens and gradients.
//
//   p[t, c] = bias[c] + sum_k w[c, k] x[t - (K-1) + k, c],   y = p or silu(p)
//   dp = dy act'(p);  dx[t] = sum_k w[k] dp[t + (K-1) - k];
//   dw[k] = sum_t dp[t] x[t - (K-1) + k];  dbias = sum_t dp[t]
//
// K <= 4 products per element against 2 to 6 bytes of traffic: memory bounds
// it.  A thread walks a piece of rows of V adjacent channels with the last K - 1
// rows in registers, so each row is loaded once per piece and only K - 1 rows per
// piece are read twice.  At 8 x 4096 x 2048 bf16, four taps: 268 MB in 56 us, 4.8
// TB/s (a large copy: 5.1); gradients 403 MB in 92.8 us, 4.3 TB/s, where forming
// p, its slope, dx and the five sums (32 operations an element) keeps the vector
// units busy three quarters of the time.
#include <algorithm>

#include "gdr2_layer.h"

namespace gdr2 {

namespace {

// Rows of V channels loaded together (>= K), so that enough bytes are in flight.
// Forwards 8 (8 x 4096 x 2048 bf16: 57 us, with 4 rows 60); backwards, where two
// row arrays are loaded and the next rows too, 8 of single channels (41.4 us for
// 10007 x 1003 fp32 rows, with 4 44.1) and 4 of wider ones (8 there take all the
// registers: 95 us against 92.8 at 8 x 4096 x 2048).
constexpr int kForwardRows = 8;
template <int V> constexpr int kBackwardRows = V == 1 ? 8 : 4;

template <typename T, int V, int K>
__device__ __forceinline__ void load_taps(const float* weight, const float* bias, int64_t c0, float (&w)[K][V], float (&b)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            w[k][v] = weight[(c0 + v) * K + k];
        b[v] = bias ? bias[c0 + v] : 0.f;
    }
}

// Row t of (state, sequence), t >= -(K-1): the raw elements, zero outside.
template <typename T, int V, int K>
__device__ __forceinline__ typename Raw<T, V>::Type conv_row(const T* x, int64_t ld, const T* state, int64_t C, int64_t t,
                                                             int64_t len)
{
    if (t >= 0)
        return t < len ? Raw<T, V>::load(x + t * ld) : Raw<T, V>::zero();
    return state ? Raw<T, V>::load(state + (t + K - 1) * C) : Raw<T, V>::zero();
}

template <typename T, int V, int K>
__global__ __launch_bounds__(256) void conv_forward_kernel(gdr2_conv_args a, Pieces pc, uint32_t ncv)
{
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    const uint32_t slot = item / ncv;
    if (slot >= pc.slots())
        return;
    const Piece q = piece_of(pc, slot);
    if (q.seq < 0)
        return;
    const int64_t C = a.C, c0 = (int64_t)(item - slot * ncv) * V;
    float w[K][V], b[V];
    load_taps<T, V, K>(a.weight, a.bias, c0, w, b);
    const T* x = (const T*)a.x + q.row0 * a.x_stride + c0;
    const T* state = a.state0 ? (const T*)a.state0 + q.seq * (K - 1) * C + c0 : nullptr;
    T* y = (T*)a.y + q.row0 * C + c0;
    const int64_t t0 = q.index << pc.lg;
    const int64_t t1 = min(q.len, t0 + ((int64_t)1 << pc.lg));

    float win[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        Raw<T, V>::get(conv_row<T, V, K>(x, a.x_stride, state, C, t0 - (K - 1) + j, q.len), win[j]);
    // the final state belongs to piece 0, which has read state0 above (the
    // two may be the same buffer): all of its rows are read before any is written
    if (q.index == 0 && a.state_out) {
        typename Raw<T, V>::Type last[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            last[j] = conv_row<T, V, K>(x, a.x_stride, state, C, q.len - (K - 1) + j, q.len);
        T* so = (T*)a.state_out + q.seq * (K - 1) * C + c0;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            *reinterpret_cast<typename Raw<T, V>::Type*>(so + j * C) = last[j];
    }
    for (int64_t t = t0; t < t1; t += kForwardRows) {
        typename Raw<T, V>::Type raw[kForwardRows];
#pragma unroll
        for (int u = 0; u < kForwardRows; ++u)
            raw[u] = t + u < t1 ? Raw<T, V>::load(x + (t + u) * a.x_stride) : Raw<T, V>::zero();
#pragma unroll
        for (int u = 0; u < kForwardRows; ++u) {
            float xv[V], o[V];
            Raw<T, V>::get(raw[u], xv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p = b[v];
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
                    p = fmaf(w[k][v], win[k][v], p);
                p = fmaf(w[K - 1][v], xv[v], p);
                o[v] = a.act == GDR2_ACT_SILU ? silu_f(p) : p;
#pragma unroll
                for (int k = 0; k < K - 2; ++k)
                    win[k][v] = win[k + 1][v];
                win[K - 2][v] = xv[v];
            }
            if (t + u < t1)
                store_row<V>(y + (t + u) * C, o);
        }
    }
}

// One token: a thread per sequence and vector of channels.  256 sequences of 2048
// bf16 channels, 8.4 MB, take 4.2 us, about a launch.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void conv_step_kernel(gdr2_conv_step_args a, uint32_t ncv)
{
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    const uint32_t n = item / ncv;
    if (n >= a.N)
        return;
    const int64_t C = a.C, c0 = (int64_t)(item - n * ncv) * V;
    T* state = (T*)a.state + (int64_t)n * (K - 1) * C + c0;
    typename Raw<T, V>::Type raw[K];
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        raw[k] = Raw<T, V>::load(state + k * C);
    raw[K - 1] = Raw<T, V>::load((const T*)a.x + (int64_t)n * a.x_stride + c0);
    float w[K][V], p[V];
    load_taps<T, V, K>(a.weight, a.bias, c0, w, p);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float xv[V];
        Raw<T, V>::get(raw[k], xv);
#pragma unroll
        for (int v = 0; v < V; ++v)
            p[v] = fmaf(w[k][v], xv[v], p[v]);
        if (k > 0)
            *reinterpret_cast<typename Raw<T, V>::Type*>(state + (k - 1) * C) = raw[k];
    }
    if (a.act == GDR2_ACT_SILU) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            p[v] = silu_f(p[v]);
    }
    store_row<V>((T*)a.y + (int64_t)n * C + c0, p);
}

// Workgroup: 2^lw channel vectors x 256 / 2^lw pieces.  Every thread sums its
// piece's share of dw and dbias in registers; the workgroup's pieces are added
// in LDS in piece order and one row of partial sums [C][K+1] leaves per
// workgroup, which the column sum adds in workgroup order.
template <typename T, int V, int K>
__global__ __launch_bounds__(256) void conv_backward_kernel(gdr2_conv_bwd_args a, Pieces pc, uint32_t ncv, int lw,
                                                            uint32_t ncb, float* part)
{
    constexpr int ROWS = kBackwardRows<V>;
    __shared__ float s_red[256 * V];
    const uint32_t rows_per = 256u >> lw;
    const uint32_t pb = blockIdx.x / ncb;                      // piece block
    const uint32_t cv = (blockIdx.x - pb * ncb) * (1u << lw) + (threadIdx.x & ((1u << lw) - 1));
    const int64_t slot = (int64_t)pb * rows_per + (threadIdx.x >> lw);
    const int64_t C = a.C, c0 = (int64_t)cv * V;
    float acc[K + 1][V] = {};
    Piece q;
    q.seq = -1;
    if (cv < ncv && slot < pc.slots())
        q = piece_of(pc, slot);
    if (q.seq >= 0) {
        float w[K][V], b[V];
        load_taps<T, V, K>(a.weight, a.bias, c0, w, b);
        const T* x = (const T*)a.x + q.row0 * a.x_stride + c0;
        const T* state = a.state0 ? (const T*)a.state0 + q.seq * (K - 1) * C + c0 : nullptr;
        const T* dst = a.dstate ? (const T*)a.dstate + q.seq * (K - 1) * C + c0 : nullptr;
        const T* dy = (const T*)a.dy + q.row0 * C + c0;
        T* dx = (T*)a.dx + q.row0 * C + c0;
        T* ds = a.dstate0 ? (T*)a.dstate0 + q.seq * (K - 1) * C + c0 : nullptr;
        const int64_t t0 = q.index << pc.lg;
        const int64_t t1 = min(q.len, t0 + ((int64_t)1 << pc.lg));
        float win[K - 1][V], dpw[K - 1][V] = {};
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            Raw<T, V>::get(conv_row<T, V, K>(x, a.x_stride, state, C, t0 - (K - 1) + j, q.len), win[j]);
        // rows t0 .. t1 + K-2: the K - 1 beyond the piece only feed its dx
        const int64_t end = t1 + K - 1, exist = min(q.len, end);
        typename Raw<T, V>::Type nx[ROWS], nd[ROWS];
        auto fetch = [&](int64_t t) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                const bool in = t + u < exist;
                nx[u] = in ? Raw<T, V>::load(x + (t + u) * a.x_stride) : Raw<T, V>::zero();
                nd[u] = in ? Raw<T, V>::load(dy + (t + u) * C) : Raw<T, V>::zero();
            }
        };
        fetch(t0);
        for (int64_t t = t0; t < end; t += ROWS) {
            typename Raw<T, V>::Type rx[ROWS], rd[ROWS];
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                rx[u] = nx[u];
                rd[u] = nd[u];
            }
            fetch(t + ROWS);
#pragma unroll
            for (int u = 0; u < ROWS; ++u) {
                float xv[V], dv[V], o[V];
                Raw<T, V>::get(rx[u], xv);
                Raw<T, V>::get(rd[u], dv);
                const bool mine = t + u < t1, exists = t + u < q.len;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float dp = dv[v];
                    if (a.act == GDR2_ACT_SILU) {
                        float p = b[v];
#pragma unroll
                        for (int k = 0; k < K - 1; ++k)
                            p = fmaf(w[k][v], win[k][v], p);
                        p = fmaf(w[K - 1][v], xv[v], p);
                        dp *= silu_slope_f(p);
                    }
                    dp = exists ? dp : 0.f;
                    // (under the test: a row that is not this piece's may hold an inf)
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < K - 1; ++k)
                            acc[k][v] = fmaf(dp, win[k][v], acc[k][v]);
                        acc[K - 1][v] = fmaf(dp, xv[v], acc[K - 1][v]);
                        acc[K][v] += dp;
                    }
                    // dx of row t + u - (K-1): taps K-1 .. 0 meet dp of rows t+u-(K-1) .. t+u
                    float g = w[0][v] * dp;
#pragma unroll
                    for (int k = 0; k < K - 1; ++k)
                        g = fmaf(w[K - 1 - k][v], dpw[k][v], g);
                    o[v] = g;
#pragma unroll
                    for (int k = 0; k < K - 2; ++k) {
                        win[k][v] = win[k + 1][v];
                        dpw[k][v] = dpw[k + 1][v];
                    }
                    win[K - 2][v] = xv[v];
                    dpw[K - 2][v] = dp;
                }
                // the rows before a sequence are its state's
                const int64_t r = t + u - (K - 1);
                T* to = r >= t0 && r < t1 ? dx + r * C : r < 0 && ds && t + u < end ? ds + (r + K - 1) * C : nullptr;
                if (to) {
                    const int64_t back = r - (q.len - (K - 1));      // the row of the final state it is, if >= 0
                    if (dst && back >= 0) {
                        float e[V];
                        Raw<T, V>::get(Raw<T, V>::load(dst + back * C), e);
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            o[v] += e[v];
                    }
                    store_row<V>(to, o);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v)
            s_red[v * 256 + threadIdx.x] = acc[k][v];
        __syncthreads();
        // column (lane, v) of this tap: the pieces' sums in piece order
        for (uint32_t m = threadIdx.x; m < (uint32_t)V << lw; m += 256) {
            const uint32_t v = m >> lw, l = m & ((1u << lw) - 1);
            float s = 0.f;
            for (uint32_t r = 0; r < rows_per; ++r)
                s += s_red[v * 256 + (r << lw) + l];
            const uint32_t c = ((blockIdx.x - pb * ncb) * (1u << lw) + l) * V + v;
            if (c < C)
                part[(int64_t)pb * C * (K + 1) + (k < K ? (int64_t)c * K + k : C * K + c)] = s;
        }
    }
}

// ---------------------------------------------------------------------------
// Column sums.  A workgroup owns 64 columns; its 4 or 16 waves take every 4th
// or 16th partial row and are added in wave order.  The latency of a wave's rows
// in turn is the time, so many rows get 16 waves: 512 rows of 4096 columns 4.9 us
// (with 4 waves 6.6); the launch of larger workgroups costs more than that saves
// on 64 rows (0.6 us).
template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void column_sum_kernel(const float* part, int64_t P, int64_t ld, int64_t M, ColumnOut a,
                                                                ColumnOut b, ColumnOut c)
{
    __shared__ float s_sum[WAVES][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (m < M) {
#pragma unroll 8
        for (int64_t p = wave; p < P; p += WAVES)
            s += part[p * ld + m];
    }
    s_sum[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || m >= M)
        return;
#pragma unroll
    for (int k = 1; k < WAVES; ++k)
        s += s_sum[k][lane];
    if (m < a.n) {
        if (a.p)
            a.p[m] = s;
    } else if (m < a.n + b.n) {
        if (b.p)
            b.p[m - a.n] = s;
    } else if (c.p) {
        c.p[m - a.n - b.n] = s;
    }
}

int64_t items_of(int64_t B, int64_t T, int64_t ncv, bool packed, int lg)
{
    const int64_t none[1] = {};
    Pieces p{packed ? none : nullptr, B, T, lg};
    return p.slots() * ncv;
}

// Rows of one piece, fewer (down to 8) while that leaves threads below two waves
// per SIMD.  Forwards 64 at most (8 x 4096 x 2048 bf16: 56.1 us; 32 rows 56.9, 16
// rows 60), backwards 128 (with four waves per SIMD asked for instead of two, and so
// 64 rows: 108 us against 92.8).
int piece_lg(int lg, int64_t B, int64_t T, int64_t ncv, bool packed)
{
    const int64_t want = (int64_t)device_cu_count() * 4 * 2 * 64;
    while (lg > 3 && items_of(B, T, ncv, packed, lg) < want)
        --lg;
    return lg;
}
constexpr int kForwardLg = 6, kBackwardLg = 7;

struct BackwardPlan {
    bool vec;
    int64_t ncv, ncb, npb;
    int lw, lg;
};

// Channels of a thread when rows are aligned to them.  Eight of bf16 (16 bytes)
// take 48.5 us against 49.8 forwards at 8 x 4096 x 2048 (one input over and over,
// part of it in the memory-side cache), but 123 against 92.1 backwards, where the
// taps, windows and sums of eight channels leave one wave per SIMD.
constexpr int kVec = 4;

bool conv_vec(const void* x, int64_t x_stride, int64_t C, int32_t dtype)
{
    return rows_aligned(x, x_stride, C, dtype == GDR2_BF16 ? 2 : 4, kVec);
}

// The workspace query sees no pointers, so its size takes the larger of the
// two channel-vector widths' plans.
BackwardPlan backward_plan(const gdr2_conv_bwd_args& a, bool vec)
{
    BackwardPlan p;
    p.vec = vec;
    p.ncv = vec ? a.C / kVec : a.C;
    p.lw = 3;
    while (p.lw < 6 && ((int64_t)1 << p.lw) < p.ncv)
        ++p.lw;
    p.ncb = ceil_div(p.ncv, (int64_t)1 << p.lw);
    p.lg = piece_lg(kBackwardLg, a.B, a.T, p.ncv, a.offsets != nullptr);
    Pieces pc{a.offsets, a.B, a.T, p.lg};
    p.npb = ceil_div(pc.slots(), 256 >> p.lw);
    return p;
}

template <typename T, int V>
hipError_t forward_k(const gdr2_conv_args& a, hipStream_t stream)
{
    const int64_t ncv = a.C / V;
    const int lg = piece_lg(kForwardLg, a.B, a.T, ncv, a.offsets != nullptr);
    const Pieces pc{a.offsets, a.B, a.T, lg};
    const dim3 grid((unsigned)ceil_div(pc.slots() * ncv, 256));
    switch (a.width) {
    case 2: hipLaunchKernelGGL((conv_forward_kernel<T, V, 2>), grid, dim3(256), 0, stream, a, pc, (uint32_t)ncv); break;
    case 3: hipLaunchKernelGGL((conv_forward_kernel<T, V, 3>), grid, dim3(256), 0, stream, a, pc, (uint32_t)ncv); break;
    default: hipLaunchKernelGGL((conv_forward_kernel<T, V, 4>), grid, dim3(256), 0, stream, a, pc, (uint32_t)ncv); break;
    }
    return hipGetLastError();
}

template <typename T, int V>
hipError_t step_k(const gdr2_conv_step_args& a, hipStream_t stream)
{
    const int64_t ncv = a.C / V;
    const dim3 grid((unsigned)ceil_div(a.N * ncv, 256));
    switch (a.width) {
    case 2: hipLaunchKernelGGL((conv_step_kernel<T, V, 2>), grid, dim3(256), 0, stream, a, (uint32_t)ncv); break;
    case 3: hipLaunchKernelGGL((conv_step_kernel<T, V, 3>), grid, dim3(256), 0, stream, a, (uint32_t)ncv); break;
    default: hipLaunchKernelGGL((conv_step_kernel<T, V, 4>), grid, dim3(256), 0, stream, a, (uint32_t)ncv); break;
    }
    return hipGetLastError();
}

template <typename T, int V>
hipError_t backward_k(const gdr2_conv_bwd_args& a, const BackwardPlan& p, hipStream_t stream)
{
    const Pieces pc{a.offsets, a.B, a.T, p.lg};
    const dim3 grid((unsigned)(p.ncb * p.npb));
    float* part = (float*)a.workspace;
    if (p.npb > 0) switch (a.width) {
    case 2: hipLaunchKernelGGL((conv_backward_kernel<T, V, 2>), grid, dim3(256), 0, stream, a, pc, (uint32_t)p.ncv, p.lw, (uint32_t)p.ncb, part); break;
    case 3: hipLaunchKernelGGL((conv_backward_kernel<T, V, 3>), grid, dim3(256), 0, stream, a, pc, (uint32_t)p.ncv, p.lw, (uint32_t)p.ncb, part); break;
    default: hipLaunchKernelGGL((conv_backward_kernel<T, V, 4>), grid, dim3(256), 0, stream, a, pc, (uint32_t)p.ncv, p.lw, (uint32_t)p.ncb, part); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    return launch_column_sum(part, p.npb, a.C * (a.width + 1), {a.dweight, a.C * a.width}, {a.dbias, a.C}, {nullptr, 0}, stream);
}

}  // namespace

hipError_t launch_column_sum(const float* part, int64_t P, int64_t ld, ColumnOut a, ColumnOut b, ColumnOut c,
                             hipStream_t stream)
{
    const int64_t M = a.n + b.n + c.n;
    const dim3 grid((unsigned)ceil_div(M, 64));
    if (P >= 256)
        hipLaunchKernelGGL(column_sum_kernel<16>, grid, dim3(1024), 0, stream, part, P, ld, M, a, b, c);
    else
        hipLaunchKernelGGL(column_sum_kernel<4>, grid, dim3(256), 0, stream, part, P, ld, M, a, b, c);
    return hipGetLastError();
}

namespace {

// Workgroups of 256 items for pieces of at most 2^lg rows; kMaxGroups stands for
// that many and for more.  (Sizes up to 2^40 each: their product is taken in
// floating point first, and below the bound every later one fits int64.)
int64_t piece_groups(int lg, int64_t B, int64_t T, int64_t ncv, bool packed)
{
    const double L = (double)((int64_t)1 << lg), b = (double)B, pieces = (double)T / L;
    const double slots = packed ? pieces + b : b * (pieces < 1.0 ? 1.0 : pieces);
    if (slots * (double)ncv >= (double)kMaxGroups * 256.0)
        return kMaxGroups;
    return std::min(kMaxGroups, ceil_div(items_of(B, T, ncv, packed, piece_lg(lg, B, T, ncv, packed)), 256));
}

}  // namespace

int64_t conv_forward_groups(const gdr2_conv_args& a)
{
    return piece_groups(kForwardLg, a.B, a.T, conv_vec(a.x, a.x_stride, a.C, a.dtype) ? a.C / kVec : a.C, a.offsets != nullptr);
}

int64_t conv_step_groups(const gdr2_conv_step_args& a)
{
    return piece_groups(kForwardLg, a.N, 1, conv_vec(a.x, a.x_stride, a.C, a.dtype) ? a.C / kVec : a.C, false);
}

// The larger of the two plans (the workspace query sees no pointers).
int64_t conv_backward_groups(const gdr2_conv_bwd_args& a)
{
    int64_t n = 0;
    for (const bool vec : {false, true}) {
        if (vec && a.C % kVec)
            continue;
        if (piece_groups(kBackwardLg, a.B, a.T, vec ? a.C / kVec : a.C, a.offsets != nullptr) >= kMaxGroups)
            return kMaxGroups;
        const BackwardPlan p = backward_plan(a, vec);
        n = std::max(n, p.ncb * p.npb);
    }
    return n;
}

hipError_t launch_conv_forward(const gdr2_conv_args& a, hipStream_t stream)
{
    const bool vec = conv_vec(a.x, a.x_stride, a.C, a.dtype);
    if (a.dtype == GDR2_BF16)
        return vec ? forward_k<bf16, kVec>(a, stream) : forward_k<bf16, 1>(a, stream);
    return vec ? forward_k<float, kVec>(a, stream) : forward_k<float, 1>(a, stream);
}

hipError_t launch_conv_step(const gdr2_conv_step_args& a, hipStream_t stream)
{
    const bool vec = conv_vec(a.x, a.x_stride, a.C, a.dtype);
    if (a.dtype == GDR2_BF16)
        return vec ? step_k<bf16, kVec>(a, stream) : step_k<bf16, 1>(a, stream);
    return vec ? step_k<float, kVec>(a, stream) : step_k<float, 1>(a, stream);
}

size_t conv_backward_workspace_bytes(const gdr2_conv_bwd_args& a)
{
    int64_t rows = backward_plan(a, false).npb;
    if (a.C % kVec == 0)
        rows = std::max(rows, backward_plan(a, true).npb);
    return (size_t)rows * a.C * (a.width + 1) * sizeof(float);
}

hipError_t launch_conv_backward(const gdr2_conv_bwd_args& a, hipStream_t stream)
{
    const BackwardPlan p = backward_plan(a, conv_vec(a.x, a.x_stride, a.C, a.dtype));
    if (a.dtype == GDR2_BF16)
        return p.vec ? backward_k<bf16, kVec>(a, p, stream) : backward_k<bf16, 1>(a, p, stream);
    return p.vec ? backward_k<float, kVec>(a, p, stream) : backward_k<float, 1>(a, p, stream);
}

}  // namespace gdr2
