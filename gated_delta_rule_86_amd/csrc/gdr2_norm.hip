// gdr2_norm.hip -- layer norm and rms norm of rows, with an optional silu
// gate, and their gradients.
//
//   xh = (x - m) r,  r = (mean((x - m)^2) + eps)^(-1/2),  m = mean or 0
//   n = xh weight + bias;   y = n, or n silu(z)
// Gradients, with dn = dy (times silu(z)) and v = dn weight:
//   dx = r (v - mean(v) [layer only] - xh mean(v xh)),
//   dz = dy n silu'(z),  dweight = sum_rows dn xh,  dbias = sum_rows dn
//
// Memory bounds both.  A row is held in registers by a group of LPR lanes
// (8 .. 64 of a wave, or a whole workgroup of 256), NV vectors of V elements
// each, so it is read once; mean and variance are two passes over those
// registers (no E[x^2] - m^2 cancellation), sums in fp32.  A group keeps its
// share of the weights in registers and walks rows g, g + groups, ..., with the
// next row's loads in flight while it works on one.  In bf16: 524288 gated rows of
// 128, 403 MB, in 75 us, 5.4 TB/s (a large copy: 5.1); layer norm's gradients of
// 32768 rows of 2048, 403 MB, in 81.7 us, 4.9 TB/s, 4.8 us of it the column sums;
// those of 524288 gated rows of 128, 671 MB, in 127 us, 5.3 TB/s.
#include <algorithm>

#include "gdr2_layer.h"

namespace gdr2 {

namespace {

// Workgroup of a kernel whose groups have LPR lanes.
template <int LPR> constexpr int kThreads = LPR > 256 ? LPR : 256;

// Sum over the LPR lanes that hold one row; every lane gets it.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* s_part)
{
    v = lanes_sum<(LPR < 64 ? LPR : 64)>(v);
    if constexpr (LPR > 64) {
        __syncthreads();                       // the previous sum has been read
        if ((threadIdx.x & 63) == 0)
            s_part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = s_part[0];
#pragma unroll
        for (int k = 1; k < LPR / 64; ++k)
            v += s_part[k];
    }
    return v;
}

// Two sums at once.
template <int LPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* s_part)
{
    a = lanes_sum<(LPR < 64 ? LPR : 64)>(a);
    b = lanes_sum<(LPR < 64 ? LPR : 64)>(b);
    if constexpr (LPR > 64) {
        constexpr int W = LPR / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            s_part[threadIdx.x >> 6] = a;
            s_part[W + (threadIdx.x >> 6)] = b;
        }
        __syncthreads();
        a = s_part[0];
        b = s_part[W];
#pragma unroll
        for (int k = 1; k < W; ++k) {
            a += s_part[k];
            b += s_part[W + k];
        }
    }
}

// A group's share of one row array, unconverted; nothing is read past C or R.
template <typename T, int V, int LPR, int NV> struct RowRegs {
    typename Raw<T, V>::Type raw[NV];
    __device__ __forceinline__ void load(const void* base, int64_t row, int64_t stride, int64_t C, int lane, bool on)
    {
        const T* p = (const T*)base + row * stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = ((int64_t)j * LPR + lane) * V;
            raw[j] = on && c < C ? Raw<T, V>::load(p + c) : Raw<T, V>::zero();
        }
    }
};

// Mean (0 for rms) and 1/rms of the row in x (elements past C are zero and
// `in` is false for their vectors).
template <int LPR, int V, int NV>
__device__ __forceinline__ void row_stats(const float (&x)[NV][V], const bool (&in)[NV], int64_t C, int kind, float eps,
                                          float* s_part, float& mean, float& rstd)
{
    const float inv = 1.f / (float)C;
    mean = 0.f;
    if (kind == GDR2_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v)
                s += x[j][v];
        mean = row_sum<LPR>(s, s_part) * inv;
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float d = in[j] ? x[j][v] - mean : 0.f;
            ss = fmaf(d, d, ss);
        }
    rstd = 1.f / sqrtf(row_sum<LPR>(ss, s_part) * inv + eps);
}

template <int V, int LPR, int NV>
__device__ __forceinline__ void group_params(const float* p, float without, int64_t C, int lane, float (&out)[NV][V])
{
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = ((int64_t)j * LPR + lane) * V;
#pragma unroll
        for (int v = 0; v < V; ++v)
            out[j][v] = p && c < C ? p[c + v] : without;
    }
}

template <typename T, int V, int LPR, int NV, bool GATE>
__global__ __launch_bounds__(256) void norm_forward_kernel(gdr2_norm_args a)
{
    __shared__ float s_part[8];
    constexpr int RPB = 256 / LPR;
    const int lane = threadIdx.x % LPR;
    const int64_t step = (int64_t)gridDim.x * RPB;
    float w[NV][V], b[NV][V];
    bool in[NV];
    group_params<V, LPR, NV>(a.weight, 1.f, a.C, lane, w);
    group_params<V, LPR, NV>(a.bias, 0.f, a.C, lane, b);
#pragma unroll
    for (int j = 0; j < NV; ++j)
        in[j] = ((int64_t)j * LPR + lane) * V < a.C;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    RowRegs<T, V, LPR, NV> nx, nz;
    nx.load(a.x, row, a.x_stride, a.C, lane, row < a.R);
    if constexpr (GATE)
        nz.load(a.z, row, a.z_stride, a.C, lane, row < a.R);
    for (; row < a.R; row += step) {          // LPR = 256: the same rows in every lane
        const RowRegs<T, V, LPR, NV> cx = nx, cz = nz;
        nx.load(a.x, row + step, a.x_stride, a.C, lane, row + step < a.R);
        if constexpr (GATE)
            nz.load(a.z, row + step, a.z_stride, a.C, lane, row + step < a.R);
        float x[NV][V], mean, rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            Raw<T, V>::get(cx.raw[j], x[j]);
        row_stats<LPR, V, NV>(x, in, a.C, a.kind, a.eps, s_part, mean, rstd);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!in[j])
                continue;
            float o[V], z[V];
            if constexpr (GATE)
                Raw<T, V>::get(cz.raw[j], z);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = fmaf((x[j][v] - mean) * rstd, w[j][v], b[j][v]);
                if constexpr (GATE)
                    o[v] *= silu_f(z[v]);
            }
            store_row<V>((T*)a.y + row * a.C + ((int64_t)j * LPR + lane) * V, o);
        }
    }
}

// Sums over a whole workgroup, for rows read in passes.
__device__ __forceinline__ float block_sum(float v, float* s_part) { return row_sum<256>(v, s_part); }

template <typename T>
__device__ __forceinline__ void looped_stats(const T* x, int64_t C, int kind, float eps, float* s_part, float& mean, float& rstd)
{
    const float inv = 1.f / (float)C;
    mean = 0.f;
    if (kind == GDR2_NORM_LAYER) {
        float s = 0.f;
        for (int64_t c = threadIdx.x; c < C; c += 256)
            s += to_f32(x[c]);
        mean = block_sum(s, s_part) * inv;
    }
    float ss = 0.f;
    for (int64_t c = threadIdx.x; c < C; c += 256) {
        const float d = to_f32(x[c]) - mean;
        ss = fmaf(d, d, ss);
    }
    rstd = 1.f / sqrtf(block_sum(ss, s_part) * inv + eps);
}

// Rows too long for the registers of a workgroup: passes over the row, which
// the caches hold.
template <typename T>
__global__ __launch_bounds__(256) void norm_forward_long_kernel(gdr2_norm_args a)
{
    __shared__ float s_part[8];
    const int64_t row = blockIdx.x;
    const T* x = (const T*)a.x + row * a.x_stride;
    float mean, rstd;
    looped_stats<T>(x, a.C, a.kind, a.eps, s_part, mean, rstd);
    for (int64_t c = threadIdx.x; c < a.C; c += 256) {
        float o = fmaf((to_f32(x[c]) - mean) * rstd, a.weight ? a.weight[c] : 1.f, a.bias ? a.bias[c] : 0.f);
        if (a.z)
            o *= silu_f(to_f32(((const T*)a.z)[row * a.z_stride + c]));
        ((T*)a.y)[row * a.C + c] = from_f32<T>(o);
    }
}

// A group's sums of dweight and dbias stay in registers, are added over the
// workgroup's groups in LDS (in group order), and leave as one row [2][C] of
// partial sums.
template <typename T, int V, int LPR, int NV, bool GATE>
__global__ __launch_bounds__(kThreads<LPR>, 2) void norm_backward_kernel(gdr2_norm_bwd_args p, float* part)
{
    const gdr2_norm_args& a = p.f;
    __shared__ float s_part[16];
    constexpr int RPB = kThreads<LPR> / LPR;
    __shared__ float s_red[RPB > 1 ? 256 * NV * V : 1];
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const float inv = 1.f / (float)a.C;
    // the weights stay in registers where they fit beside the sums and the loads
    constexpr bool HOLD = NV * V <= 16 || !GATE;
    float dw[NV][V] = {}, db[NV][V] = {}, wr[HOLD ? NV : 1][V];
    bool in[NV];
    if constexpr (HOLD)
        group_params<V, LPR, NV>(a.weight, 1.f, a.C, lane, wr);
#pragma unroll
    for (int j = 0; j < NV; ++j)
        in[j] = ((int64_t)j * LPR + lane) * V < a.C;
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    RowRegs<T, V, LPR, NV> nx, nd, nz;
    auto fetch = [&](int64_t r) {
        nx.load(a.x, r, a.x_stride, a.C, lane, r < a.R);
        nd.load(p.dy, r, a.C, a.C, lane, r < a.R);
        if constexpr (GATE)
            nz.load(a.z, r, a.z_stride, a.C, lane, r < a.R);
    };
    fetch(row);
    for (; row < a.R; row += step) {
        float x[NV][V], g[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            Raw<T, V>::get(nx.raw[j], x[j]);
            Raw<T, V>::get(nd.raw[j], g[j]);
        }
        const RowRegs<T, V, LPR, NV> cz = nz;
        fetch(row + step);
        float mean, rstd;
        row_stats<LPR, V, NV>(x, in, a.C, a.kind, a.eps, s_part, mean, rstd);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!in[j])
                continue;
            const int64_t c = ((int64_t)j * LPR + lane) * V;
            float z[V], dz[V];
            if constexpr (GATE)
                Raw<T, V>::get(cz.raw[j], z);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xh = (x[j][v] - mean) * rstd;
                const float w = HOLD ? wr[HOLD ? j : 0][v] : a.weight ? a.weight[c + v] : 1.f;
                float dn = g[j][v];
                if constexpr (GATE) {
                    const float b = a.bias ? a.bias[c + v] : 0.f, sg = sigmoid_f(z[v]);
                    dz[v] = dn * fmaf(xh, w, b) * (sg * fmaf(z[v], 1.f - sg, 1.f));
                    dn *= z[v] * sg;
                }
                dw[j][v] = fmaf(dn, xh, dw[j][v]);
                db[j][v] += dn;
                const float e = dn * w;
                s1 += e;
                s2 = fmaf(e, xh, s2);
                x[j][v] = xh;
                g[j][v] = e;
            }
            if constexpr (GATE)
                store_row<V>((T*)p.dz + row * a.C + c, dz);
        }
        row_sum2<LPR>(s1, s2, s_part);
        const float m1 = a.kind == GDR2_NORM_LAYER ? s1 * inv : 0.f, m2 = s2 * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!in[j])
                continue;
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                o[v] = rstd * (g[j][v] - m1 - x[j][v] * m2);
            store_row<V>((T*)p.dx + row * a.C + ((int64_t)j * LPR + lane) * V, o);
        }
    }
    if (!part)
        return;
    float* to = part + (int64_t)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if constexpr (RPB == 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (in[j])
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        to[half * a.C + ((int64_t)j * LPR + lane) * V + v] = half ? db[j][v] : dw[j][v];
        } else {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s_red[grp * (LPR * NV * V) + (j * LPR + lane) * V + v] = half ? db[j][v] : dw[j][v];
            __syncthreads();
            for (int c = threadIdx.x; c < a.C; c += 256) {
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < RPB; ++r)
                    s += s_red[r * (LPR * NV * V) + c];
                to[half * a.C + c] = s;
            }
        }
    }
}

// Long rows, backwards: one workgroup per row writes dx and dz in passes and
// leaves the row's mean and 1/rms for the column pass.
template <typename T>
__global__ __launch_bounds__(256) void norm_backward_long_kernel(gdr2_norm_bwd_args p, float* stats)
{
    const gdr2_norm_args& a = p.f;
    __shared__ float s_part[8];
    const int64_t row = blockIdx.x;
    const float inv = 1.f / (float)a.C;
    const T* x = (const T*)a.x + row * a.x_stride;
    const T* dy = (const T*)p.dy + row * a.C;
    const T* z = a.z ? (const T*)a.z + row * a.z_stride : nullptr;
    float mean, rstd;
    looped_stats<T>(x, a.C, a.kind, a.eps, s_part, mean, rstd);
    if (threadIdx.x == 0) {
        stats[2 * row] = mean;
        stats[2 * row + 1] = rstd;
    }
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < a.C; c += 256) {
        const float w = a.weight ? a.weight[c] : 1.f, xh = (to_f32(x[c]) - mean) * rstd;
        float dn = to_f32(dy[c]);
        if (z) {
            const float zc = to_f32(z[c]);
            ((T*)p.dz)[row * a.C + c] = from_f32<T>(dn * fmaf(xh, w, a.bias ? a.bias[c] : 0.f) * silu_slope_f(zc));
            dn *= silu_f(zc);
        }
        s1 += dn * w;
        s2 = fmaf(dn * w, xh, s2);
    }
    row_sum2<256>(s1, s2, s_part);
    const float m1 = a.kind == GDR2_NORM_LAYER ? s1 * inv : 0.f, m2 = s2 * inv;
    for (int64_t c = threadIdx.x; c < a.C; c += 256) {
        const float w = a.weight ? a.weight[c] : 1.f, xh = (to_f32(x[c]) - mean) * rstd;
        float dn = to_f32(dy[c]);
        if (z)
            dn *= silu_f(to_f32(z[c]));
        ((T*)p.dx)[row * a.C + c] = from_f32<T>(rstd * (dn * w - m1 - xh * m2));
    }
}

// dweight and dbias of long rows: a workgroup sums 64 columns, a wave every
// fourth row of every gridDim.y-th block of four.
template <typename T>
__global__ __launch_bounds__(256) void norm_backward_columns_kernel(gdr2_norm_bwd_args p, const float* stats, float* part)
{
    const gdr2_norm_args& a = p.f;
    __shared__ float s_red[2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float dw = 0.f, db = 0.f;
    if (c < a.C) {
        for (int64_t row = (int64_t)blockIdx.y * 4 + wave; row < a.R; row += (int64_t)gridDim.y * 4) {
            const float xh = (to_f32(((const T*)a.x)[row * a.x_stride + c]) - stats[2 * row]) * stats[2 * row + 1];
            float dn = to_f32(((const T*)p.dy)[row * a.C + c]);
            if (a.z)
                dn *= silu_f(to_f32(((const T*)a.z)[row * a.z_stride + c]));
            dw = fmaf(dn, xh, dw);
            db += dn;
        }
    }
    s_red[0][wave][lane] = dw;
    s_red[1][wave][lane] = db;
    __syncthreads();
    if (wave < 2 && c < a.C)
        part[(int64_t)blockIdx.y * 2 * a.C + wave * a.C + c] =
            (s_red[wave][0][lane] + s_red[wave][1][lane]) + (s_red[wave][2][lane] + s_red[wave][3][lane]);
}

// ---- variants --------------------------------------------------------------
// The narrowest group of lanes whose registers hold the row: a wave, or part
// of one, while a lane has at most 32 elements; backwards, where a lane also
// holds dy, dweight, dbias and the next row's loads, 32 in bf16 without a gate
// and 16 otherwise.  Then a workgroup of 256 with up to 64 elements a lane
// forwards and 16 backwards, backwards one of 512, then passes over the row.
// (More elements backwards spill: 8192 columns on 256 lanes kept 130 to 1200
// bytes a lane in scratch.)
struct Shape {
    int lpr, nv;   // lpr == 0: passes
};

Shape shape_of(int64_t C, int V, bool backward, bool gate)
{
    const int64_t nvec = (C + V - 1) / V;
    for (int lpr = 8; lpr <= 64; lpr *= 2)
        if (nvec <= lpr)
            return {lpr, 1};
    const int wave = V == 1 ? 8 : backward && (V == 4 || gate) ? 16 / V : 32 / V;
    for (int nv = 2; nv <= wave; nv *= 2)
        if (nvec <= 64 * nv)
            return {64, nv};
    const int most = backward ? 16 / V : V == 1 ? 32 : 64 / V;
    for (int nv = 1; nv <= most; nv *= 2)
        if (nvec <= 256 * nv)
            return {256, nv};
    if (backward && nvec <= 512 * most)
        return {512, most};
    return {0, 0};
}

#define GDR2_NORM_CASE(L, N)                                                                     \
    if (s.lpr == L && s.nv == N) {                                                               \
        f.template operator()<L, N>();                                                           \
        return hipGetLastError();                                                                \
    }

template <typename T, int V> struct ForwardLaunch {
    const gdr2_norm_args& a;
    hipStream_t stream;
    template <int L, int N> void operator()() const
    {
        // eight workgroups per compute unit, then the rows are walked
        const dim3 grid((unsigned)std::min(ceil_div(a.R, 256 / L), (int64_t)device_cu_count() * 8));
        if (a.z)
            hipLaunchKernelGGL((norm_forward_kernel<T, V, L, N, true>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((norm_forward_kernel<T, V, L, N, false>), grid, dim3(256), 0, stream, a);
    }
};

template <typename T, int V, bool GATE> struct BackwardLaunch {
    const gdr2_norm_bwd_args& p;
    float* part;
    int64_t groups;
    hipStream_t stream;
    template <int L, int N> void operator()() const
    {
        hipLaunchKernelGGL((norm_backward_kernel<T, V, L, N, GATE>), dim3((unsigned)groups), dim3(kThreads<L>), 0, stream, p,
                           part);
    }
};

// Exactly the shapes shape_of can return for V forwards ..
template <int V, typename F> hipError_t dispatch_forward(const Shape& s, const F& f)
{
    GDR2_NORM_CASE(8, 1) GDR2_NORM_CASE(16, 1) GDR2_NORM_CASE(32, 1) GDR2_NORM_CASE(64, 1)
    GDR2_NORM_CASE(64, 2) GDR2_NORM_CASE(64, 4) GDR2_NORM_CASE(256, 4) GDR2_NORM_CASE(256, 8)
    if constexpr (V == 8) {
        GDR2_NORM_CASE(256, 2)
    } else {
        GDR2_NORM_CASE(64, 8) GDR2_NORM_CASE(256, 16)
    }
    if constexpr (V == 1) {
        GDR2_NORM_CASE(256, 32)
    }
    return hipErrorInvalidValue;
}

// .. and backwards.
template <int V, bool GATE, typename F> hipError_t dispatch_backward(const Shape& s, const F& f)
{
    GDR2_NORM_CASE(8, 1) GDR2_NORM_CASE(16, 1) GDR2_NORM_CASE(32, 1) GDR2_NORM_CASE(64, 1) GDR2_NORM_CASE(64, 2)
    if constexpr (V == 8) {
        if constexpr (GATE) {
            GDR2_NORM_CASE(256, 1)
        } else {
            GDR2_NORM_CASE(64, 4)
        }
        GDR2_NORM_CASE(256, 2) GDR2_NORM_CASE(512, 2)
    } else if constexpr (V == 4) {
        GDR2_NORM_CASE(64, 4) GDR2_NORM_CASE(256, 2) GDR2_NORM_CASE(256, 4) GDR2_NORM_CASE(512, 4)
    } else {
        GDR2_NORM_CASE(64, 4) GDR2_NORM_CASE(64, 8) GDR2_NORM_CASE(256, 4) GDR2_NORM_CASE(256, 8) GDR2_NORM_CASE(256, 16)
        GDR2_NORM_CASE(512, 16)
    }
    return hipErrorInvalidValue;
}

bool norm_vec(const gdr2_norm_args& a)
{
    const int64_t e = a.dtype == GDR2_BF16 ? 2 : 4;
    const int V = (int)(16 / e);
    return rows_aligned(a.x, a.x_stride, a.C, e, V) && (!a.z || rows_aligned(a.z, a.z_stride, a.C, e, V));
}

template <typename T, int V>
hipError_t forward_v(const gdr2_norm_args& a, hipStream_t stream)
{
    const Shape s = shape_of(a.C, V, false, a.z);
    if (s.lpr == 0) {
        hipLaunchKernelGGL((norm_forward_long_kernel<T>), dim3((unsigned)a.R), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    return dispatch_forward<V>(s, ForwardLaunch<T, V>{a, stream});
}

// Workgroups of the backward: two per compute unit, fewer when there are
// fewer rows.
int64_t backward_groups(int64_t R, const Shape& s)
{
    return std::min(ceil_div(R, std::max(1, 256 / s.lpr)), (int64_t)device_cu_count() * 2);
}

int64_t long_row_blocks(int64_t R, int64_t C)
{
    return std::max((int64_t)1, std::min(ceil_div(R, 4), (int64_t)device_cu_count() * 4 / ceil_div(C, 64)));
}

template <typename T, int V>
hipError_t backward_v(const gdr2_norm_bwd_args& p, hipStream_t stream)
{
    const gdr2_norm_args& a = p.f;
    const Shape s = shape_of(a.C, V, true, a.z);
    const bool sums = p.dweight || p.dbias;
    float* part = (float*)p.workspace;
    int64_t P = 0;
    if (a.R == 0) {
        // nothing but the sums' zeros to write
    } else if (s.lpr != 0) {
        P = backward_groups(a.R, s);
        float* to = sums ? part : nullptr;
        const hipError_t e = a.z ? dispatch_backward<V, true>(s, BackwardLaunch<T, V, true>{p, to, P, stream})
                                 : dispatch_backward<V, false>(s, BackwardLaunch<T, V, false>{p, to, P, stream});
        if (e != hipSuccess || !sums)
            return e;
    } else {
        float* stats = part;
        part += 2 * a.R;
        P = long_row_blocks(a.R, a.C);
        hipLaunchKernelGGL((norm_backward_long_kernel<T>), dim3((unsigned)a.R), dim3(256), 0, stream, p, stats);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !sums)
            return e;
        hipLaunchKernelGGL((norm_backward_columns_kernel<T>), dim3((unsigned)ceil_div(a.C, 64), (unsigned)P), dim3(256), 0,
                           stream, p, stats, part);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return sums ? launch_column_sum(part, P, 2 * a.C, {p.dweight, a.C}, {p.dbias, a.C}, {nullptr, 0}, stream) : hipSuccess;
}

}  // namespace

// Workgroups of a call's largest launch: rows held in registers are walked by a
// few per compute unit, longer ones take one each.  (Backwards for either width
// of access: the workspace query sees no pointers.)
int64_t norm_launch_groups(const gdr2_norm_args& a, bool backward)
{
    const int wide = a.dtype == GDR2_BF16 ? 8 : 4;
    bool whole = shape_of(a.C, backward || !norm_vec(a) ? 1 : wide, backward, a.z).lpr != 0;
    if (backward)
        whole = whole && shape_of(a.C, wide, backward, a.z).lpr != 0;
    return whole ? std::min(a.R, (int64_t)device_cu_count() * 8) : a.R;
}

hipError_t launch_norm_forward(const gdr2_norm_args& a, hipStream_t stream)
{
    if (a.dtype == GDR2_BF16)
        return norm_vec(a) ? forward_v<bf16, 8>(a, stream) : forward_v<bf16, 1>(a, stream);
    return norm_vec(a) ? forward_v<float, 4>(a, stream) : forward_v<float, 1>(a, stream);
}

// The larger of the vector and the scalar variant's needs (the query sees no
// pointers).
size_t norm_backward_workspace_bytes(const gdr2_norm_bwd_args& p)
{
    const gdr2_norm_args& a = p.f;
    int64_t floats = 0;
    for (int V : {1, a.dtype == GDR2_BF16 ? 8 : 4}) {
        const Shape s = shape_of(a.C, V, true, a.z);
        floats = std::max(floats, s.lpr ? backward_groups(a.R, s) * 2 * a.C : 2 * a.R + long_row_blocks(a.R, a.C) * 2 * a.C);
    }
    return (size_t)floats * sizeof(float);
}

hipError_t launch_norm_backward(const gdr2_norm_bwd_args& p, hipStream_t stream)
{
    if (p.f.dtype == GDR2_BF16)
        return norm_vec(p.f) ? backward_v<bf16, 8>(p, stream) : backward_v<bf16, 1>(p, stream);
    return norm_vec(p.f) ? backward_v<float, 4>(p, stream) : backward_v<float, 1>(p, stream);
}

}  // namespace gdr2
