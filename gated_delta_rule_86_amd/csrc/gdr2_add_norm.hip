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
// to 1024), one or two vectors of eight elements each, read once; the next
// row's loads are in flight while one is worked on.  A row's sums are fp64
// (squares of fp32 numbers pass fp32's range), and forwards so is n: a code next
// to a rounding border is then the same however the row is spread over lanes.
// An fp64 operation costs this chip's vector units what one of fp32 does:
// forwards that is hidden, in the gradients the sums' longer way over the lanes
// is 4 us of 111 (32768 rows of 2048).  There the forward with h and y takes
// 113 us (4.7 TB/s; a large copy 5.15), with h and an 8-bit y 105, the gradients
// 111 (4.8 TB/s), from rows in 8 bits 104; 1 row 15 us, all of it the call.
#include <algorithm>

#include "gdr2_block.h"
#include "gdr2_scan.h"

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
// Sum over aligned groups of W lanes.
template <int W> __device__ __forceinline__ double wave_sum(double v)
{
    static_assert(W == 4 || W == 16 || W == 64, "lanes");
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    if constexpr (W >= 16) {
        v += dpp_move<0x141>(v);
        v += dpp_move<0x140>(v);
    }
    if constexpr (W >= 64)
        v = swap_sum32(swap_sum16(v));
    return v;
}

// N sums over the LPR lanes that hold one row; every lane gets them.  Over
// more than a wave they go through one of two places in turn: one barrier a
// sum, for a place is written again behind the next one's.
template <int LPR, int N> struct RowSums {
    static constexpr int W = LPR > 64 ? LPR / 64 : 1;
    typedef double Place[2][W][N];
    Place* place;
    int turn = 0;
    __device__ __forceinline__ explicit RowSums(Place* p) : place(p) {}
    template <int M> __device__ __forceinline__ void operator()(double (&v)[M])
    {
        static_assert(M <= N, "place");
#pragma unroll
        for (int i = 0; i < M; ++i)
            v[i] = wave_sum<(LPR < 64 ? LPR : 64)>(v[i]);
        if constexpr (LPR > 64) {
            if ((threadIdx.x & 63) == 0)
#pragma unroll
                for (int i = 0; i < M; ++i)
                    (*place)[turn][threadIdx.x >> 6][i] = v[i];
            lds_barrier();
#pragma unroll
            for (int i = 0; i < M; ++i)
                v[i] = wave_sum<W>((*place)[turn][threadIdx.x % W][i]);
            turn ^= 1;
        }
    }
};

template <int LPR> constexpr int kThreads = LPR > 256 ? LPR : 256;
// Whether the next row's loads, and the weights, fit the registers (a workgroup
// of 1024 has 128 a lane); elsewhere both are loaded where they are used, the
// vectors one after the other (4096 rows of 16384, gradients: held, with many spills,
// 231 us, loaded again, with 2 to 15 registers spilled, 141).
template <int LPR, int NV> constexpr bool kRoomy = LPR * NV < 2048;

// x^(-1/2): the unit's estimate and two Newton steps, each doubling its bits;
// infinite for 0 and 0 for infinity (the steps would make NaN of both).
__device__ __forceinline__ double inverse_root(double x)
{
    const double first = __builtin_amdgcn_rsq(x);
    double y = first;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        y = fma(y, fma(-0.5 * x * y, y, 0.5), y);
    return x > 0.0 && x < __builtin_inf() ? y : first;
}

// The element's 64-bit value as fp32 bits for a rounding to fewer bits: the
// leading 21 bits, and a last one that is set if any bit behind them is.  A
// conversion to fp32 and then to e4m3 would round twice.
__device__ __forceinline__ uint32_t sticky_bits(double v)
{
    const uint32_t hi = (uint32_t)__double2hiint(v), lo = (uint32_t)__double2loint(v), mag = hi & 0x7fffffffu;
    const uint32_t bits = ((mag - (896u << 20)) << 3) | (lo != 0 ? 1u : 0u) | (hi & 0x80000000u);
    const bool normal = mag - (897u << 20) < (254u << 20);
    return __builtin_unpredictable(normal) ? bits : __builtin_bit_cast(uint32_t, (float)v);
}

// A group's share of one row array.  TAIL: the row ends within a vector.
// Otherwise lanes past its end read its last vector, and rows past the last one
// the last one: no branch; what they hold goes into no sum and is not written.
template <typename T, int NV, bool TAIL> struct RowRegs {
    Row8<T> part[NV];
    template <int LPR> __device__ __forceinline__ void load(const void* base, int64_t row, int64_t R, int64_t stride, int C, int lane)
    {
        const T* p = (const T*)base + (row < R ? row : R - 1) * stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * 8;
            if constexpr (TAIL)
                part[j].load(p + c, C - c);
            else
                part[j].load(p + min(c, C - 8));
        }
    }
};

// Weights or biases of a vector, n of whose elements exist.
__device__ __forceinline__ void params(const float* p, float without, int c, int n, float (&out)[8])
{
#pragma unroll
    for (int v = 0; v < 8; ++v)
        out[v] = without;
    if (p && n > 0) {
        Row8<float> r;
        r.load(p + c, n);
        r.get(out);
    }
}

// A lane's weights: held, or loaded for each row.
template <int LPR, int NV> struct Weights {
    const float* p;
    int lane, C;
    float held[kRoomy<LPR, NV> ? NV : 1][8];
    __device__ __forceinline__ Weights(const float* p_, int lane_, int C_) : p(p_), lane(lane_), C(C_)
    {
        if constexpr (kRoomy<LPR, NV>)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                load(j, held[j]);
    }
    __device__ __forceinline__ void load(int j, float (&w)[8]) const { params(p, 1.f, (j * LPR + lane) * 8, C - (j * LPR + lane) * 8, w); }
    __device__ __forceinline__ void get(int j, float (&w)[8]) const
    {
        if constexpr (kRoomy<LPR, NV>) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                w[v] = held[j][v];
        } else {
            load(j, w);
        }
    }
};

// A vector's codes and its block's scale, for the lanes of a block together.
struct Vector8 {
    Codes8 codes;
    int e;
    __device__ __forceinline__ Vector8(const float (&v)[8], int n)
    {
        const int amax = block_max<8>(v, n);
        e = block_exponent(amax);
        codes.pack(v, amax, e);
    }
    __device__ __forceinline__ void store(const gdr2_rows8& to, int64_t row, int C, int64_t blocks, int c, int n) const
    {
        codes.store((uint8_t*)to.codes + row * C + c, n);
        if (c % kRows8 == 0)
            ((uint8_t*)to.scales)[row * blocks + c / kRows8] = (uint8_t)(e + 127);
    }
};

// ---- forward ---------------------------------------------------------------
template <typename TX, typename TR, int LPR, int NV, bool TAIL>
__global__ __launch_bounds__(kThreads<LPR>) void add_norm_forward_kernel(gdr2_add_norm_args a)
{
    typedef RowSums<LPR, 1> Sums;
    __shared__ typename Sums::Place s_part;
    Sums sums(&s_part);
    constexpr int RPB = kThreads<LPR> / LPR;
    const int lane = threadIdx.x % LPR, C = (int)a.C;
    const int64_t step = (int64_t)gridDim.x * RPB, blocks = scale_count(C);
    const double inv = 1.0 / (double)C;
    Weights<LPR, NV> weights(a.weight, lane, C);
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    RowRegs<TX, NV, TAIL> nx;
    RowRegs<TR, NV, TAIL> nr;
    auto fetch = [&](int64_t r) {
        nx.template load<LPR>(a.x, r, a.R, a.x_stride, C, lane);
        if (a.residual)
            nr.template load<LPR>(a.residual, r, a.R, a.res_stride, C, lane);
    };
    if constexpr (kRoomy<LPR, NV>)
        fetch(row);
    // every lane of a workgroup goes as often
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.R; first += step, row += step) {
        if constexpr (!kRoomy<LPR, NV>)
            fetch(row);
        float h[NV][8];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx.part[j].get(h[j]);
            if (a.residual) {
                float r[8];
                nr.part[j].get(r);
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    h[j][v] = to_f32(from_f32<TR>(h[j][v] + r[v]));
            }
#pragma unroll
            for (int v = 0; v < 8; ++v)
                here(h[j][v]);
        }
        if constexpr (kRoomy<LPR, NV>)
            fetch(row + step);
        double mean = 0.0;
        if (a.kind == GDR2_NORM_LAYER) {
            double s[1] = {0.0};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int n = C - (j * LPR + lane) * 8;
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    s[0] += (double)(v < n ? h[j][v] : 0.f);
            }
            sums(s);
            mean = s[0] * inv;
        }
        double ss[1] = {0.0};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int n = C - (j * LPR + lane) * 8;
            double part = 0.0;
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const double d = (double)h[j][v] - mean;
                part = TAIL && v >= n ? part : fma(d, d, part);
            }
            ss[0] += n > 0 ? part : 0.0;
        }
        sums(ss);
        const double rstd = inverse_root(ss[0] * inv + (double)a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * 8, n = row < a.R ? C - c : 0;
#pragma unroll
            for (int v = 0; v < 8; ++v)
                here(h[j][v]);
            if (a.h && n > 0)
                Row8<TR>::store((TR*)a.h + row * C + c, h[j], n);
            if (a.h8.codes) {
                const Vector8 k(h[j], n);
                if (n > 0)
                    k.store(a.h8, row, C, blocks, c, n);
            }
            if (!a.y && !a.y8.codes)
                continue;
            float w[8], b[8] = {}, y[8], y8[8];
            weights.get(j, w);
            if (a.bias)
                params(a.bias, 0.f, c, C - c, b);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                here(w[v]);
                const double t = fma(((double)h[j][v] - mean) * rstd, (double)w[v], (double)b[v]);
                y[v] = (float)t;
                y8[v] = __builtin_bit_cast(float, sticky_bits(t));
            }
            if (a.y && n > 0)
                Row8<TX>::store((TX*)a.y + row * C + c, y, n);
            if (a.y8.codes) {
                const Vector8 k(y8, n);
                if (n > 0)
                    k.store(a.y8, row, C, blocks, c, n);
            }
            if constexpr (!kRoomy<LPR, NV>)
                __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// ---- gradients -------------------------------------------------------------
// The stream's rows as they are, or in 8 bits.
template <typename TR, bool P8, int NV, bool TAIL> struct StreamRegs {
    RowRegs<TR, NV, TAIL> rows;
    template <int LPR> __device__ __forceinline__ void load(const gdr2_add_norm_bwd_args& a, int64_t row, int lane)
    {
        rows.template load<LPR>(a.h, row, a.R, a.C, (int)a.C, lane);
    }
    __device__ __forceinline__ void get(int j, float (&v)[8]) const { rows.part[j].get(v); }
};
template <typename TR, int NV, bool TAIL> struct StreamRegs<TR, true, NV, TAIL> {
    Codes8 codes[NV];
    uint32_t scale[NV];
    template <int LPR> __device__ __forceinline__ void load(const gdr2_add_norm_bwd_args& a, int64_t row, int lane)
    {
        const int64_t from = row < a.R ? row : a.R - 1, nb = scale_count(a.C);
        const int C = (int)a.C;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int own = (j * LPR + lane) * 8, c = TAIL ? min(own, C - 1) : min(own, C - 8);
            codes[j].load((const uint8_t*)a.h8.codes + from * C + c, TAIL ? C - own : 8);
            scale[j] = ((const uint8_t*)a.h8.scales)[from * nb + c / kRows8];
        }
    }
    __device__ __forceinline__ void get(int j, float (&v)[8]) const { codes[j].get(scale[j], v); }
};

// A group's sums of dweight and dbias stay in registers, are added over the
// workgroup's groups in LDS (in group order), and leave as one row [2][C] of
// partial sums.
template <typename TX, typename TR, bool P8, int LPR, int NV, bool TAIL>
__global__ __launch_bounds__(kThreads<LPR>) void add_norm_backward_kernel(gdr2_add_norm_bwd_args a, float* part)
{
    typedef RowSums<LPR, 3> Sums;
    __shared__ typename Sums::Place s_part;
    Sums sums(&s_part);
    constexpr int RPB = kThreads<LPR> / LPR;
    __shared__ float s_red[RPB > 1 ? 256 * NV * 8 : 1];
    const int lane = threadIdx.x % LPR, grp = threadIdx.x / LPR, C = (int)a.C;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const double inv = 1.0 / (double)C;
    float dw[NV][8] = {}, db[NV][8] = {};
    Weights<LPR, NV> weights(a.weight, lane, C);
    int64_t row = (int64_t)blockIdx.x * RPB + grp;
    StreamRegs<TR, P8, NV, TAIL> nh;
    RowRegs<TX, NV, TAIL> nd;
    auto fetch = [&](int64_t r) {
        nh.template load<LPR>(a, r, lane);
        nd.template load<LPR>(a.dy, r, a.R, C, C, lane);
    };
    if constexpr (kRoomy<LPR, NV>)
        fetch(row);
    for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.R; first += step, row += step) {
        if constexpr (!kRoomy<LPR, NV>)
            fetch(row);
        float x[NV][8], g[NV][8];
        RowRegs<TR, NV, TAIL> dh;
        if (kRoomy<LPR, NV> && a.dh)
            dh.template load<LPR>(a.dh, row, a.R, C, C, lane);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nh.get(j, x[j]);
            nd.part[j].get(g[j]);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                here(x[j][v]);
                here(g[j][v]);
            }
        }
        if constexpr (kRoomy<LPR, NV>)
            fetch(row + step);
        double mean = 0.0;
        if (a.kind == GDR2_NORM_LAYER) {
            double s[1] = {0.0};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int n = C - (j * LPR + lane) * 8;
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    s[0] += (double)(v < n ? x[j][v] : 0.f);
            }
            sums(s);
            mean = s[0] * inv;
        }
        // sum d^2, sum v d and, for the layer norm, sum v, in one go: xh = r d
        double s[3] = {0.0, 0.0, 0.0};
        float sv = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            // elements and rows that are not there add nothing, whatever they hold
            const int n = row < a.R ? C - (j * LPR + lane) * 8 : 0;
            float w[8];
            weights.get(j, w);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const bool in = TAIL ? v < n : n > 0;
                const float d = in ? (float)((double)x[j][v] - mean) : 0.f;
                x[j][v] = d;
                g[j][v] = in ? g[j][v] : 0.f;
                const float gw = g[j][v] * w[v];
                s[0] = fma((double)d, (double)d, s[0]);
                s[1] = fma((double)gw, (double)d, s[1]);
                sv += gw;
            }
            if constexpr (!kRoomy<LPR, NV>)
                __builtin_amdgcn_sched_barrier(0);
        }
        if (a.kind == GDR2_NORM_LAYER) {
            s[2] = (double)sv;
            sums(s);
        } else {
            double two[2] = {s[0], s[1]};
            sums(two);
            s[0] = two[0];
            s[1] = two[1];
        }
        const double root = inverse_root(s[0] * inv + (double)a.eps);
        const float rstd = (float)root;
        const float m1 = a.kind == GDR2_NORM_LAYER ? (float)(s[2] * inv) : 0.f, m2 = (float)(root * s[1] * inv);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LPR + lane) * 8, n = row < a.R ? C - c : 0;
            float w[8], o[8], more[8] = {};
            weights.get(j, w);
            if (!kRoomy<LPR, NV> && a.dh)
                dh.template load<LPR>(a.dh, row, a.R, C, C, lane);
            if (a.dh)
                dh.part[j].get(more);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                // (a row that is not there has d = 0, and may have an infinite r)
                const float xh = n > 0 ? x[j][v] * rstd : 0.f;
                dw[j][v] = fmaf(g[j][v], xh, dw[j][v]);
                db[j][v] += g[j][v];
                o[v] = fmaf(rstd, fmaf(g[j][v], w[v], -m1) - xh * m2, more[v]);
            }
            if (n > 0 && a.dresidual)
                Row8<TR>::store((TR*)a.dresidual + row * C + c, o, n);
            if (n > 0 && a.dx)
                Row8<TX>::store((TX*)a.dx + row * C + c, o, n);
            if constexpr (!kRoomy<LPR, NV>)
                __builtin_amdgcn_sched_barrier(0);
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
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    if ((j * LPR + lane) * 8 + v < C)
                        to[half * C + (j * LPR + lane) * 8 + v] = half ? db[j][v] : dw[j][v];
        } else {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    s_red[grp * (LPR * NV * 8) + (j * LPR + lane) * 8 + v] = half ? db[j][v] : dw[j][v];
            __syncthreads();
            for (int c = threadIdx.x; c < C; c += 256) {
                float s = 0.f;
#pragma unroll
                for (int r = 0; r < RPB; ++r)
                    s += s_red[r * (LPR * NV * 8) + c];
                to[half * C + c] = s;
            }
        }
    }
}

// ---- variants --------------------------------------------------------------
// The narrowest group of lanes whose registers hold the row with at most two
// vectors each: part of a wave, a wave, a workgroup of 256, one of 1024.  (Four
// vectors a lane take 256 registers, one wave a SIMD: 32768 rows of 2048 with an
// 8-bit output in 153 us.)
struct Shape {
    int lpr, nv;
};
constexpr int kLanes[] = {16, 64, 256, 1024};

Shape shape_of(int64_t C)
{
    const int64_t vectors = ceil_div(C, 8);
    for (int lpr : kLanes)
        for (int nv = 1; nv <= (lpr == 16 ? 1 : 2); ++nv)
            if (vectors <= lpr * nv)
                return {lpr, nv};
    return {0, 0};           // refused before
}

#define GDR2_ADD_NORM_CASE(L, N)                                                                 \
    if (s.lpr == L && s.nv == N) {                                                               \
        f.template operator()<L, N>();                                                           \
        return hipGetLastError();                                                                \
    }

template <typename F> hipError_t dispatch(const Shape& s, const F& f)
{
    GDR2_ADD_NORM_CASE(16, 1) GDR2_ADD_NORM_CASE(64, 1) GDR2_ADD_NORM_CASE(64, 2) GDR2_ADD_NORM_CASE(256, 1)
    GDR2_ADD_NORM_CASE(256, 2) GDR2_ADD_NORM_CASE(1024, 1) GDR2_ADD_NORM_CASE(1024, 2)
    return hipErrorInvalidValue;
}

template <typename TX, typename TR> struct ForwardLaunch {
    const gdr2_add_norm_args& a;
    hipStream_t stream;
    template <int L, int N> void operator()() const
    {
        // eight workgroups of 256 per compute unit (as many waves in larger ones), then the rows are walked
        constexpr int RPB = kThreads<L> / L;
        const dim3 grid((unsigned)std::min(ceil_div(a.R, RPB), (int64_t)device_cu_count() * 2048 / kThreads<L>));
        if (a.C % 8)
            hipLaunchKernelGGL((add_norm_forward_kernel<TX, TR, L, N, true>), grid, dim3(kThreads<L>), 0, stream, a);
        else
            hipLaunchKernelGGL((add_norm_forward_kernel<TX, TR, L, N, false>), grid, dim3(kThreads<L>), 0, stream, a);
    }
};

template <typename TX, typename TR, bool P8> struct BackwardLaunch {
    const gdr2_add_norm_bwd_args& a;
    float* part;
    int64_t groups;
    hipStream_t stream;
    template <int L, int N> void operator()() const
    {
        const dim3 grid((unsigned)groups);
        if (a.C % 8)
            hipLaunchKernelGGL((add_norm_backward_kernel<TX, TR, P8, L, N, true>), grid, dim3(kThreads<L>), 0, stream, a, part);
        else
            hipLaunchKernelGGL((add_norm_backward_kernel<TX, TR, P8, L, N, false>), grid, dim3(kThreads<L>), 0, stream, a, part);
    }
};

// Workgroups of the gradients, each of which leaves a row of partial sums: of
// 256 threads three per compute unit, two where a lane holds two vectors (32768
// rows of 2048: two 120 us, three 111, four 116; 16384 of 4096: two 111, three
// 117, four 127), of 1024 one; fewer when there are fewer rows.
int64_t backward_groups(const gdr2_add_norm_bwd_args& a)
{
    const Shape s = shape_of(a.C);
    const int64_t per_unit = s.lpr > 256 ? 1 : s.nv == 2 ? 2 : 3;
    return std::min(ceil_div(a.R, std::max(1, 256 / s.lpr)), device_cu_count() * per_unit);
}

template <typename TX, typename TR> hipError_t backward_p(const gdr2_add_norm_bwd_args& a, float* part, int64_t P, hipStream_t stream)
{
    return a.h ? dispatch(shape_of(a.C), BackwardLaunch<TX, TR, false>{a, part, P, stream})
               : dispatch(shape_of(a.C), BackwardLaunch<TX, TR, true>{a, part, P, stream});
}

}  // namespace

hipError_t launch_add_norm_forward(const gdr2_add_norm_args& a, hipStream_t stream)
{
    const Shape s = shape_of(a.C);
    if (a.dtype == GDR2_F32)
        return dispatch(s, ForwardLaunch<float, float>{a, stream});
    return a.res_dtype == GDR2_F32 ? dispatch(s, ForwardLaunch<bf16, float>{a, stream}) : dispatch(s, ForwardLaunch<bf16, bf16>{a, stream});
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
