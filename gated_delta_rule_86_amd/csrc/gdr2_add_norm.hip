// gdr2_add_norm.hip -- layer norm and rms norm of a residual stream, with the
// addition that makes it, an output in 8 bits and the stream in 8 bits for the
// gradients; and the gradients.
//
//   h = x + residual (rounded to the stream's type)
//   xh = (h - m) r,  r = (mean((h - m)^2) + eps)^(-1/2),  m = mean or 0
//   n = xh weight + bias;   y = n,  y8 = rows8(n),  h8 = rows8(h)
// Gradients, with v = dy weight:
//   dresidual = dx = dh + r (v - mean(v) [layer only] - xh mean(v xh))
//   dweight = sum_rows dy xh,  dbias = sum_rows dy
//
// Memory bounds both.  A row is held in registers by a group of LPR lanes (16
// to 1024), NV vectors of V elements each, read once.  Forwards the sums and n
// are fp64: a code next to a rounding border is then the same however the row
// is spread over lanes, and fp64 costs this chip's vector units what fp32
// does.
#include <algorithm>

#include "gdr2_block.h"

namespace gdr2 {

namespace {

// ---- sums over lanes -------------------------------------------------------
template <int CTRL> __device__ __forceinline__ double dpp_move(double v)
{
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, true);
    return __hiloint2double(hi, lo);
}
// The sums of lanes a row of 16, or a half of the wave, apart.
__device__ __forceinline__ double swap_sum16(double v)
{
    const auto lo = __builtin_amdgcn_permlane16_swap(__double2loint(v), __double2loint(v), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(__double2hiint(v), __double2hiint(v), false, false);
    return __hiloint2double(hi[0], lo[0]) + __hiloint2double(hi[1], lo[1]);
}
__device__ __forceinline__ double swap_sum32(double v)
{
    const auto lo = __builtin_amdgcn_permlane32_swap(__double2loint(v), __double2loint(v), false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(__double2hiint(v), __double2hiint(v), false, false);
    return __hiloint2double(hi[0], lo[0]) + __hiloint2double(hi[1], lo[1]);
}
template <int W> __device__ __forceinline__ double wave_sum(double v)
{
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    v += dpp_move<0x141>(v);
    v += dpp_move<0x140>(v);
    if constexpr (W >= 64)
        v = swap_sum32(swap_sum16(v));
    return v;
}
template <int W> __device__ __forceinline__ float wave_sum(float v) { return lanes_sum<W>(v); }

// Sum over the LPR lanes that hold one row; every lane gets it.
template <int LPR, typename S> __device__ __forceinline__ S row_sum(S v, S* s_part)
{
    v = wave_sum<(LPR < 64 ? LPR : 64)>(v);
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

template <int LPR> constexpr int kThreads = LPR > 256 ? LPR : 256;

// The element's 64-bit value as fp32 bits for a rounding to fewer bits: the
// leading 21 bits, and a last one that is set if any bit behind them is.  A
// conversion to fp32 and then to e4m3 would round twice.
__device__ __forceinline__ uint32_t sticky_bits(double v)
{
    const uint32_t hi = (uint32_t)__double2hiint(v), lo = (uint32_t)__double2loint(v), mag = hi & 0x7fffffffu;
    const uint32_t bits = ((mag - (896u << 20)) << 3) | (lo != 0 ? 1u : 0u) | (hi & 0x80000000u);
    const bool normal = mag - (897u << 20) < (254u << 20);
    return normal ? bits : __builtin_bit_cast(uint32_t, (float)v);
}

template <typename T, int V, int NV> struct RowRegs {
    RowPart<T, V> part[NV];
    template <int LPR> __device__ __forceinline__ void load(const void* base, int64_t row, int64_t stride, int C, int lane, bool on)
    {
        const T* p = (const T*)base + row * stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * V;
            if (on && c < C)
                part[j].load(p + c);
            else
                part[j].zero();
        }
    }
};

template <int V> __device__ __forceinline__ void params(const float* p, float without, int c, bool in, float (&out)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        out[v] = p && in ? p[c + v] : without;
}

// The lanes of a block (those past the row's end among them) write its V codes
// each, the first of them the scale.
template <int V>
__device__ __forceinline__ void put_rows8(const gdr2_rows8& to, int64_t row, int C, int c, const float (&v)[V], bool in)
{
    const int64_t nb = scale_count(C);
    const int amax = block_max<V>(v, in), e = block_exponent(amax);
    Codes<V> k;
    k.pack(v, amax, e);
    if (in) {
        k.store((uint8_t*)to.codes + row * C + c);
        if (c % kRows8 == 0)
            ((uint8_t*)to.scales)[row * nb + c / kRows8] = (uint8_t)(e + 127);
    }
}

// ---- forward ---------------------------------------------------------------
template <typename TX, typename TR, int V, int LPR, int NV>
__global__ __launch_bounds__(kThreads<LPR>) void add_norm_forward_kernel(gdr2_add_norm_args a)
{
    __shared__ double s_part[LPR > 64 ? LPR / 64 : 1];
    constexpr int RPB = kThreads<LPR> / LPR;
    constexpr bool HOLD = LPR < 1024;          // parameters and the next row's loads in registers
    const int lane = threadIdx.x % LPR, C = (int)a.C;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const double inv = 1.0 / (double)C;
    float w[HOLD ? NV : 1][V], b[HOLD ? NV : 1][V];
    if constexpr (HOLD) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * V;
            params<V>(a.weight, 1.f, c, c < C, w[j]);
            params<V>(a.bias, 0.f, c, c < C, b[j]);
        }
    }
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    RowRegs<TX, V, NV> nx;
    RowRegs<TR, V, NV> nr;
    auto fetch = [&](int64_t r) {
        nx.template load<LPR>(a.x, r, a.x_stride, C, lane, r < a.R);
        if (a.residual)
            nr.template load<LPR>(a.residual, r, a.res_stride, C, lane, r < a.R);
    };
    if constexpr (HOLD)
        fetch(row);
    // every lane of a workgroup goes as often: rows past the last one are zero, and not written
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.R; first += step, row += step) {
        if constexpr (!HOLD)
            fetch(row);
        const bool on = row < a.R;
        float h[NV][V];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx.part[j].get(h[j]);
            if (a.residual) {
                float r[V];
                nr.part[j].get(r);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    h[j][v] = to_f32(from_f32<TR>(h[j][v] + r[v]));
            }
        }
        if constexpr (HOLD)
            fetch(row + step);
        double mean = 0.0;
        if (a.kind == GDR2_NORM_LAYER) {
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s += (double)h[j][v];
            mean = row_sum<LPR>(s, s_part) * inv;
        }
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = (j * LPR + lane) * V < C;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const double d = in ? (double)h[j][v] - mean : 0.0;
                ss = fma(d, d, ss);
            }
        }
        const double rstd = 1.0 / sqrt(row_sum<LPR>(ss, s_part) * inv + (double)a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * V;
            const bool in = on && c < C;
            if (a.h && in)
                RowPart<TR, V>::store((TR*)a.h + row * C + c, h[j]);
            if (a.h8.codes)
                put_rows8<V>(a.h8, row, C, c, h[j], in);
            if (!a.y && !a.y8.codes)
                continue;
            float wj[V], bj[V], n[V], n8[V];
            if constexpr (!HOLD) {
                params<V>(a.weight, 1.f, c, c < C, wj);
                params<V>(a.bias, 0.f, c, c < C, bj);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const double t = fma(((double)h[j][v] - mean) * rstd, (double)(HOLD ? w[HOLD ? j : 0][v] : wj[v]),
                                     (double)(HOLD ? b[HOLD ? j : 0][v] : bj[v]));
                n[v] = (float)t;
                n8[v] = __builtin_bit_cast(float, sticky_bits(t));
            }
            if (a.y && in)
                RowPart<TX, V>::store((TX*)a.y + row * C + c, n);
            if (a.y8.codes)
                put_rows8<V>(a.y8, row, C, c, n8, in);
        }
    }
}

// ---- gradients -------------------------------------------------------------
// The stream's rows as they are, or in 8 bits.
template <typename TR, bool P8, int V, int NV> struct StreamRegs {
    RowRegs<TR, V, NV> rows;
    template <int LPR> __device__ __forceinline__ void load(const gdr2_add_norm_bwd_args& a, int64_t row, int lane, bool on)
    {
        rows.template load<LPR>(a.h, row, a.C, (int)a.C, lane, on);
    }
    __device__ __forceinline__ void get(int j, float (&v)[V]) const { rows.part[j].get(v); }
};
template <typename TR, int V, int NV> struct StreamRegs<TR, true, V, NV> {
    Codes<V> codes[NV];
    uint32_t scale[NV];
    template <int LPR> __device__ __forceinline__ void load(const gdr2_add_norm_bwd_args& a, int64_t row, int lane, bool on)
    {
        const int64_t nb = scale_count(a.C);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * V;
            codes[j].zero();
            scale[j] = 127;
            if (on && c < (int)a.C) {
                codes[j].load((const uint8_t*)a.h8.codes + row * a.C + c);
                scale[j] = ((const uint8_t*)a.h8.scales)[row * nb + c / kRows8];
            }
        }
    }
    __device__ __forceinline__ void get(int j, float (&v)[V]) const { codes[j].get(scale[j], v); }
};

// A group's sums of dweight and dbias stay in registers, are added over the
// workgroup's groups in LDS (in group order), and leave as one row [2][C] of
// partial sums.
template <typename TX, typename TR, bool P8, int V, int LPR, int NV>
__global__ __launch_bounds__(kThreads<LPR>) void add_norm_backward_kernel(gdr2_add_norm_bwd_args a, float* part)
{
    __shared__ float s_part[LPR > 64 ? LPR / 64 : 1];
    constexpr int RPB = kThreads<LPR> / LPR;
    __shared__ float s_red[RPB > 1 ? 256 * NV * V : 1];
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, C = (int)a.C;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const float inv = 1.f / (float)C;
    constexpr bool HOLD = LPR < 1024;          // the next row's loads in registers
    float dw[NV][V] = {}, db[NV][V] = {};
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    StreamRegs<TR, P8, V, NV> nh;
    RowRegs<TX, V, NV> nd;
    auto fetch = [&](int64_t r) {
        nh.template load<LPR>(a, r, lane, r < a.R);
        nd.template load<LPR>(a.dy, r, C, C, lane, r < a.R);
    };
    if constexpr (HOLD)
        fetch(row);
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.R; first += step, row += step) {
        if constexpr (!HOLD)
            fetch(row);
        const bool on = row < a.R;
        float x[NV][V], g[NV][V];
        RowRegs<TR, V, NV> dh;
        if (a.dh)
            dh.template load<LPR>(a.dh, row, C, C, lane, on);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nh.get(j, x[j]);
            nd.part[j].get(g[j]);
        }
        if constexpr (HOLD)
            fetch(row + step);
        float mean = 0.f, ss = 0.f;
        if (a.kind == GDR2_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s += x[j][v];
            mean = row_sum<LPR>(s, s_part) * inv;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = (j * LPR + lane) * V < C;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[j][v] = in ? x[j][v] - mean : 0.f;
                ss = fmaf(x[j][v], x[j][v], ss);
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<LPR>(ss, s_part) * inv + a.eps);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * V;
            float w[V];
            params<V>(a.weight, 1.f, c, c < C, w);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xh = x[j][v] * rstd;
                // a row past the last one has dy = 0, but its xh may be NaN (eps = 0)
                if (on) {
                    dw[j][v] = fmaf(g[j][v], xh, dw[j][v]);
                    db[j][v] += g[j][v];
                }
                const float e = g[j][v] * w[v];
                s1 += e;
                s2 = fmaf(e, xh, s2);
                x[j][v] = xh;
                g[j][v] = e;
            }
        }
        if (a.kind == GDR2_NORM_LAYER)
            s1 = row_sum<LPR>(s1, s_part) * inv;
        else
            s1 = 0.f;
        s2 = row_sum<LPR>(s2, s_part) * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * V;
            if (!on || c >= C)
                continue;
            float o[V], more[V];
            if (a.dh)
                dh.part[j].get(more);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = rstd * (g[j][v] - s1 - x[j][v] * s2);
                if (a.dh)
                    o[v] += more[v];
            }
            if (a.dresidual)
                RowPart<TR, V>::store((TR*)a.dresidual + row * C + c, o);
            if (a.dx)
                RowPart<TX, V>::store((TX*)a.dx + row * C + c, o);
        }
    }
    if (!part)
        return;
    float* to = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if constexpr (RPB == 1) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if ((j * LPR + lane) * V < C)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        to[half * C + (j * LPR + lane) * V + v] = half ? db[j][v] : dw[j][v];
        } else {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s_red[grp * (LPR * NV * V) + (j * LPR + lane) * V + v] = half ? db[j][v] : dw[j][v];
            __syncthreads();
            for (int c = threadIdx.x; c < C; c += 256) {
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < RPB; ++r)
                    s += s_red[r * (LPR * NV * V) + c];
                to[half * C + c] = s;
            }
        }
    }
}

// ---- variants --------------------------------------------------------------
// The narrowest group of lanes whose registers hold the row: 16 lanes of one
// vector, a wave with up to 32 elements a lane, workgroups of 256 (32 elements
// forwards, 16 backwards, where a lane also holds dy, dweight and dbias) and
// 1024 lanes (16).
struct Shape {
    int lpr, nv;
};

Shape shape_of(int64_t C, int V, bool backward)
{
    const int64_t nvec = ceil_div(C, V);
    if (V == 8 && nvec <= 16)
        return {16, 1};
    const int wave = (backward ? 16 : 32) / V, group = (backward ? 16 : 32) / V;
    for (int nv = 1; nv <= wave; nv *= 2)
        if (nvec <= 64 * nv)
            return {64, nv};
    for (int nv = wave / 2; nv <= group; nv *= 2)
        if (nvec <= 256 * nv)
            return {256, nv};
    return {1024, 16 / V};
}

#define GDR2_ADD_NORM_CASE(L, N)                                                                 \
    if (s.lpr == L && s.nv == N) {                                                               \
        f.template operator()<L, N>();                                                           \
        return hipGetLastError();                                                                \
    }

// Exactly the shapes shape_of can return.
template <int V, bool BACKWARD, typename F> hipError_t dispatch(const Shape& s, const F& f)
{
    GDR2_ADD_NORM_CASE(64, 1) GDR2_ADD_NORM_CASE(64, 2)
    if constexpr (V == 8) {
        GDR2_ADD_NORM_CASE(16, 1) GDR2_ADD_NORM_CASE(256, 2) GDR2_ADD_NORM_CASE(1024, 2)
        if constexpr (BACKWARD) {
            GDR2_ADD_NORM_CASE(256, 1)
        } else {
            GDR2_ADD_NORM_CASE(64, 4) GDR2_ADD_NORM_CASE(256, 4)
        }
    } else {
        GDR2_ADD_NORM_CASE(64, 4) GDR2_ADD_NORM_CASE(64, 8) GDR2_ADD_NORM_CASE(64, 16) GDR2_ADD_NORM_CASE(256, 16)
        GDR2_ADD_NORM_CASE(1024, 16)
        if constexpr (BACKWARD) {
            GDR2_ADD_NORM_CASE(256, 8)
        } else {
            GDR2_ADD_NORM_CASE(64, 32) GDR2_ADD_NORM_CASE(256, 32)
        }
    }
    return hipErrorInvalidValue;
}

template <typename TX, typename TR, int V> struct ForwardLaunch {
    const gdr2_add_norm_args& a;
    hipStream_t stream;
    template <int L, int N> void operator()() const
    {
        // eight workgroups of 256 per compute unit, then the rows are walked
        constexpr int RPB = kThreads<L> / L;
        const dim3 grid((unsigned)std::min(ceil_div(a.R, RPB), (int64_t)device_cu_count() * 2048 / kThreads<L>));
        hipLaunchKernelGGL((add_norm_forward_kernel<TX, TR, V, L, N>), grid, dim3(kThreads<L>), 0, stream, a);
    }
};

template <typename TX, typename TR, bool P8, int V> struct BackwardLaunch {
    const gdr2_add_norm_bwd_args& a;
    float* part;
    int64_t groups;
    hipStream_t stream;
    template <int L, int N> void operator()() const
    {
        hipLaunchKernelGGL((add_norm_backward_kernel<TX, TR, P8, V, L, N>), dim3((unsigned)groups), dim3(kThreads<L>), 0, stream,
                           a, part);
    }
};

template <typename TX, typename TR> hipError_t forward_t(const gdr2_add_norm_args& a, hipStream_t stream)
{
    const bool wide = rows_in_eights(a.x, a.x_stride, a.C, a.dtype) &&
                      (!a.residual || rows_in_eights(a.residual, a.res_stride, a.C, a.res_dtype));
    if (wide)
        return dispatch<8, false>(shape_of(a.C, 8, false), ForwardLaunch<TX, TR, 8>{a, stream});
    return dispatch<1, false>(shape_of(a.C, 1, false), ForwardLaunch<TX, TR, 1>{a, stream});
}

int width_of(const gdr2_add_norm_bwd_args& a) { return a.C % 8 == 0 ? 8 : 1; }

// Workgroups of the gradients: two of 256 threads per compute unit (as many
// waves in larger ones), fewer when there are fewer rows.
int64_t backward_groups(const gdr2_add_norm_bwd_args& a)
{
    const Shape s = shape_of(a.C, width_of(a), true);
    const int64_t most = s.lpr > 256 ? device_cu_count() : (int64_t)device_cu_count() * 2;
    return std::min(ceil_div(a.R, std::max(1, 256 / s.lpr)), most);
}

template <typename TX, typename TR, bool P8> hipError_t backward_t(const gdr2_add_norm_bwd_args& a, float* part, int64_t P, hipStream_t stream)
{
    const int V = width_of(a);
    const Shape s = shape_of(a.C, V, true);
    return V == 8 ? dispatch<8, true>(s, BackwardLaunch<TX, TR, P8, 8>{a, part, P, stream})
                  : dispatch<1, true>(s, BackwardLaunch<TX, TR, P8, 1>{a, part, P, stream});
}

template <typename TX, typename TR> hipError_t backward_p(const gdr2_add_norm_bwd_args& a, float* part, int64_t P, hipStream_t stream)
{
    return a.h ? backward_t<TX, TR, false>(a, part, P, stream) : backward_t<TX, TR, true>(a, part, P, stream);
}

}  // namespace

hipError_t launch_add_norm_forward(const gdr2_add_norm_args& a, hipStream_t stream)
{
    if (a.dtype == GDR2_F32)
        return forward_t<float, float>(a, stream);
    return a.res_dtype == GDR2_F32 ? forward_t<bf16, float>(a, stream) : forward_t<bf16, bf16>(a, stream);
}

size_t add_norm_backward_workspace_bytes(const gdr2_add_norm_bwd_args& a)
{
    return a.dweight || a.dbias ? (size_t)(backward_groups(a) * 2 * a.C) * sizeof(float) : 0;
}

hipError_t launch_add_norm_backward(const gdr2_add_norm_bwd_args& a, hipStream_t stream)
{
    const bool sums = a.dweight || a.dbias;
    float* part = sums ? (float*)a.workspace : nullptr;
    const int64_t P = backward_groups(a);
    if (a.R > 0) {
        const hipError_t e = a.dtype == GDR2_F32       ? backward_p<float, float>(a, part, P, stream)
                             : a.res_dtype == GDR2_F32 ? backward_p<bf16, float>(a, part, P, stream)
                                                       : backward_p<bf16, bf16>(a, part, P, stream);
        if (e != hipSuccess)
            return e;
    }
    return sums ? launch_column_sum(part, P, 2 * a.C, {a.dweight, a.C}, {a.dbias, a.C}, {nullptr, 0}, stream) : hipSuccess;
}

}  // namespace gdr2
