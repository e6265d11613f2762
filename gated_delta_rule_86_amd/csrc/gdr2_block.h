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

// V codes (V = 1: in the low byte; V = 8: two words) of a block with exponent e.
template <int V> struct Codes {
    uint32_t w[V == 8 ? 2 : 1];
    __device__ __forceinline__ void pack(const float (&v)[V], int amax, int e)
    {
        if (__builtin_expect(amax < 0, 0)) {
            float c[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                c[i] = clip_infinity(v[i]);
            set(c, 1.f);
        } else {
            set(v, scale_of(e + 127));
        }
    }
    __device__ __forceinline__ void set(const float (&v)[V], float scale)
    {
        const s16x2 none = {0, 0};
        if constexpr (V == 8) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = __builtin_bit_cast(uint32_t, codes2<true>(v[4 * h + 2], v[4 * h + 3], scale,
                                                                codes2<false>(v[4 * h], v[4 * h + 1], scale, none)));
        } else if constexpr (V == 2) {
            w[0] = __builtin_bit_cast(uint32_t, codes2<false>(v[0], v[1], scale, none));
        } else {
            w[0] = __builtin_bit_cast(uint32_t, codes2<false>(v[0], 0.f, scale, none));
        }
    }
    __device__ __forceinline__ void load(const uint8_t* p)
    {
        if constexpr (V == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x;
            w[1] = x.y;
        } else if constexpr (V == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
            w[0] = *p;
        }
    }
    __device__ __forceinline__ void store(uint8_t* p) const
    {
        if constexpr (V == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (V == 2)
            *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
        else
            *p = (uint8_t)w[0];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (uint32_t& x : w)
            x = 0;
    }
    // values at the scale byte s
    __device__ __forceinline__ void get(uint32_t s, float (&v)[V]) const
    {
        const float scale = scale_of(s);
        if constexpr (V == 8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], scale, false);
                const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[h], scale, true);
                v[4 * h] = lo[0];
                v[4 * h + 1] = lo[1];
                v[4 * h + 2] = hi[0];
                v[4 * h + 3] = hi[1];
            }
        } else {
            const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[0], scale, false);
#pragma unroll
            for (int i = 0; i < V; ++i)
                v[i] = lo[i];
        }
    }
};

// V consecutive elements as they lie in memory.  Eight fp32 go as two accesses
// of 16 bytes, which is all the alignment their rows are asked for.
template <typename T, int V> struct RowPart {
    static constexpr int N = V == 8 ? 8 * (int)sizeof(T) / 16 : 1, W = V / N;
    typedef Raw<T, W> Part;
    typename Part::Type raw[N];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            raw[j] = Part::load(p + j * W);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            raw[j] = Part::zero();
    }
    __device__ __forceinline__ void get(float (&v)[V]) const
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            Part::get(raw[j], v + j * W);
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[V])
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            store_row<W>(p + j * W, v + j * W);
    }
};
// Whether RowPart<T, 8> can read rows of `width` elements, `stride` apart.
inline bool rows_in_eights(const void* p, int64_t stride, int64_t width, int32_t dtype)
{
    return width % 8 == 0 && rows_aligned(p, stride, width, dtype == GDR2_BF16 ? 2 : 4, dtype == GDR2_BF16 ? 8 : 4);
}

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

// Largest finite magnitude of the V values of each lane of a block's lanes.
template <int V> __device__ __forceinline__ int block_max(const float (&v)[V], bool in)
{
    int m = -1;
#pragma unroll
    for (int i = 0; i < V; ++i)
        m = max(m, finite_bits(__builtin_bit_cast(uint32_t, v[i])));
    return lanes_max<kRows8 / V>(in ? m : -1);
}

__host__ __device__ inline int64_t scale_count(int64_t C) { return (C + kRows8 - 1) / kRows8; }

}  // namespace gdr2
