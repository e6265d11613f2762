// gdr2_block.h -- shared by the block operators (rows in 8 bits, norm with the
// residual's addition, gated linear recurrence): the 8-bit format and the
// launchers' declarations.  Not part of the ABI.
#pragma once

#include "gdr2_layer.h"

namespace gdr2 {

// ---- launchers (arguments are validated; they only enqueue work) ----------
hipError_t launch_pack(const gdr2_pack_args& a, hipStream_t stream);
hipError_t launch_unpack(const gdr2_unpack_args& a, hipStream_t stream);

constexpr int64_t kAddNormMaxWidth = 16384;
hipError_t launch_add_norm_forward(const gdr2_add_norm_args& a, hipStream_t stream);
hipError_t launch_add_norm_backward(const gdr2_add_norm_bwd_args& a, hipStream_t stream);
size_t add_norm_backward_workspace_bytes(const gdr2_add_norm_bwd_args& a);

// Rows of a call are at most this far apart: offsets within a wave's rows are
// formed in 32 bits of bytes.
constexpr int64_t kGlrMaxStride = (int64_t)1 << 22;
hipError_t launch_glr_forward(const gdr2_glr_args& a, hipStream_t stream);
hipError_t launch_glr_step(const gdr2_glr_step_args& a, hipStream_t stream);
hipError_t launch_glr_backward(const gdr2_glr_bwd_args& a, hipStream_t stream);
size_t glr_workspace_bytes(const gdr2_glr_args& a);
size_t glr_backward_workspace_bytes(const gdr2_glr_bwd_args& a);
// Workgroups, counted as of 256 threads, of a call's largest launch.
int64_t glr_launch_groups(const gdr2_glr_args& a, bool backward);

// A value that is formed here: not earlier, as an invariant of a loop whose
// registers it would fill, and not later, where it is used: what it is formed
// from gives its registers to the loads that follow.
__device__ __forceinline__ void here(float& v) { asm volatile("" : "+v"(v)); }

// ---- rows in 8 bits --------------------------------------------------------
constexpr int kRows8 = GDR2_ROWS8_BLOCK;

// A magnitude as an integer that orders like it, -1 for NaN and infinities:
// the largest over a block is then -1 where it has no finite value.
__device__ __forceinline__ int finite_bits(uint32_t bits)
{
    const int m = (int)(bits & 0x7fffffffu);
    return m < 0x7f800000 ? m : -1;
}

// A block's exponent from its largest magnitude: the smallest e >= -127 with
// that <= 448 2^e.  448 is 1.75 2^8, so the exponent field, less 127 + 8, goes
// up by one where the mantissa is above 1.75 (an addition carries into it).
// A block without finite values takes 120, where +-448 overflow to infinity.
__device__ __forceinline__ int block_exponent(int amax)
{
    const int e = ((amax + 0x1fffff) >> 23) - 135;
    return amax < 0 ? 120 : max(e, -127);
}
// A scale as the scaled conversions take it: the exponent field of an fp32
// number, 0 for 2^-127.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

typedef short s16x2 __attribute__((ext_vector_type(2)));

// Two values over their block's scale as codes, in the low or high half of
// `old` (v_cvt_scalef32_pk_fp8_*): the quotient is exact, the rounding to
// nearest even, and an infinity becomes NaN.
template <bool HIGH> __device__ __forceinline__ s16x2 codes2(float a, float b, float scale, s16x2 old)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(old, a, b, scale, HIGH);
}
// For blocks without finite values: infinities as +-448, NaN as it is.
__device__ __forceinline__ float clip_infinity(float v) { return __builtin_isinf(v) ? __builtin_copysignf(448.f, v) : v; }

// V = 1 or 2 values of codes in the low bytes of w, at the scale byte s.
template <int V> __device__ __forceinline__ void values_of(uint32_t w, uint32_t s, float (&v)[V])
{
    const auto x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, scale_of(s), false);
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = x[i];
}

// ---- eight consecutive elements of a row -----------------------------------
// One or two accesses of 16 bytes (of 8 for codes) that need the alignment of
// an element only, so rows of any width and spacing go this way.  n elements
// of the eight exist: where fewer do, they go one by one.
template <typename T> struct Row8 {
    static constexpr int N = sizeof(T) == 2 ? 1 : 2, W = 8 / N;
    typedef T Part __attribute__((ext_vector_type(W), aligned(sizeof(T))));
    typedef T Vec __attribute__((ext_vector_type(W)));
    Vec raw[N];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            raw[j] = *reinterpret_cast<const Part*>(p + j * W);
    }
    __device__ __forceinline__ void load(const T* p, int n)
    {
        if (n >= 8) {
            load(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                raw[i / W][i % W] = i < n ? p[i] : (T)0.f;
        }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (float)raw[i / W][i % W];
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[8], int n)
    {
        if (n >= 8) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                Vec x;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    x[i] = (T)v[j * W + i];
                *reinterpret_cast<Part*>(p + j * W) = x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    p[i] = (T)v[i];
        }
    }
};

struct Codes8 {
    typedef uint32_t Part __attribute__((ext_vector_type(2), aligned(1)));
    uint32_t w[2];
    __device__ __forceinline__ void set(const float (&v)[8], float scale)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = __builtin_bit_cast(uint32_t, codes2<true>(v[4 * h + 2], v[4 * h + 3], scale,
                                                            codes2<false>(v[4 * h], v[4 * h + 1], scale, s16x2{0, 0})));
    }
    // of a block with this largest magnitude and exponent
    __device__ __forceinline__ void pack(const float (&v)[8], int amax, int e)
    {
        set(v, scale_of(e + 127));
        // (asked of the wave: a branch per lane would be taken apart into masks)
        if (__builtin_expect(__any(amax < 0), 0)) {
            Codes8 k;
            float c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                c[i] = clip_infinity(v[i]);
            k.set(c, 1.f);
            w[0] = amax < 0 ? k.w[0] : w[0];
            w[1] = amax < 0 ? k.w[1] : w[1];
        }
    }
    __device__ __forceinline__ void load(const uint8_t* p, int n)
    {
        if (n >= 8) {
            const Part x = *reinterpret_cast<const Part*>(p);
            w[0] = x[0];
            w[1] = x[1];
        } else {
            w[0] = w[1] = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
        }
    }
    __device__ __forceinline__ void store(uint8_t* p, int n) const
    {
        if (n >= 8) {
            *reinterpret_cast<Part*>(p) = Part{w[0], w[1]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
        }
    }
    __device__ __forceinline__ void get(uint32_t s, float (&v)[8]) const
    {
        const float scale = scale_of(s);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], scale, false);
            const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], scale, true);
            v[4 * h] = lo[0];
            v[4 * h + 1] = lo[1];
            v[4 * h + 2] = hi[0];
            v[4 * h + 3] = hi[1];
        }
    }
};

// Largest of the values of aligned groups of W lanes, in every lane.
template <int W> __device__ __forceinline__ int lanes_max(int v)
{
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true));
    v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true));
    if constexpr (W >= 8)
        v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true));
    if constexpr (W >= 16)
        v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true));
    if constexpr (W >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max((int)r[0], (int)r[1]);
    }
    return v;
}

// Largest finite magnitude of a block whose lanes hold V values each, the first
// n of which exist.
template <int V> __device__ __forceinline__ int block_max(const float (&v)[V], int n)
{
    int m = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int x = finite_bits(__builtin_bit_cast(uint32_t, v[i]));
        m = max(m, i < n ? x : -1);
    }
    return lanes_max<kRows8 / V>(m);
}

__host__ __device__ inline int64_t scale_count(int64_t C) { return (C + kRows8 - 1) / kRows8; }

}  // namespace gdr2
