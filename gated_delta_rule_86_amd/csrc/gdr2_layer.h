// gdr2_layer.h -- shared by the layer operators (convolution, scan, norm):
// the map from work slots to pieces of sequences, row access in either dtype,
// the gate functions, and the launchers' declarations.  Not part of the ABI.
#pragma once

#include "gdr2_device.h"
#include "gdr2_internal.h"

namespace gdr2 {

// ---- launchers (arguments are validated; they only enqueue work) ----------
hipError_t launch_conv_forward(const gdr2_conv_args& a, hipStream_t stream);
hipError_t launch_conv_step(const gdr2_conv_step_args& a, hipStream_t stream);
hipError_t launch_conv_backward(const gdr2_conv_bwd_args& a, hipStream_t stream);
size_t conv_backward_workspace_bytes(const gdr2_conv_bwd_args& a);
int64_t conv_forward_groups(const gdr2_conv_args& a);
int64_t conv_step_groups(const gdr2_conv_step_args& a);
int64_t conv_backward_groups(const gdr2_conv_bwd_args& a);

hipError_t launch_scan_forward(const gdr2_scan_args& a, hipStream_t stream);
hipError_t launch_scan_step(const gdr2_scan_step_args& a, hipStream_t stream);
hipError_t launch_scan_backward(const gdr2_scan_bwd_args& a, hipStream_t stream);
size_t scan_workspace_bytes(const gdr2_scan_args& a);
size_t scan_backward_workspace_bytes(const gdr2_scan_bwd_args& a);
// Workgroups, counted as of 256 threads, of a call's largest launch.
enum class ScanCall { Forward, Step, Backward };
int64_t scan_launch_groups(const gdr2_scan_args& a, ScanCall call);

hipError_t launch_norm_forward(const gdr2_norm_args& a, hipStream_t stream);
hipError_t launch_norm_backward(const gdr2_norm_bwd_args& a, hipStream_t stream);
size_t norm_backward_workspace_bytes(const gdr2_norm_bwd_args& a);
int64_t norm_launch_groups(const gdr2_norm_args& a, bool backward);

// Column sums of part [P][M] (rows ld apart), in an order fixed by P alone.  The columns are
// cut into up to three outputs (M = their n together); NULL ones are skipped.
struct ColumnOut {
    float* p;
    int64_t n;
};
hipError_t launch_column_sum(const float* part, int64_t P, int64_t ld, ColumnOut a, ColumnOut b, ColumnOut c,
                             hipStream_t stream);

constexpr int64_t kMaxGroups = (int64_t)1 << 24;   // 256-thread workgroups of one launch, exclusive

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- pieces of sequences ---------------------------------------------------
// A sequence of `len` rows is cut into pieces of L = 2^lg rows, the last one
// shorter; an empty sequence still has one (empty) piece 0, which owns its
// states.  Work slots number the pieces:
//   dense   slot = s * per + i, per = max(1, ceil(T / L));
//   packed  slot = offsets[s] / L + s + i.  Sequence s + 1 starts at or after
//           slot offsets[s]/L + ceil(len/L) + s, so pieces do not collide, and
//           floor(T/L) + B slots hold them all: the grid is known on the host
//           without reading the offsets.  Slots no piece maps to are idle.
struct Pieces {
    const int64_t* offsets;   // NULL: dense
    int64_t B, T;
    int lg;

    __host__ __device__ int64_t per() const { const int64_t n = (T + ((int64_t)1 << lg) - 1) >> lg; return n > 0 ? n : 1; }
    __host__ __device__ int64_t slots() const { return offsets && B > 0 ? (T >> lg) + B : B * per(); }
};

struct Piece {
    int64_t seq;     // -1: an idle slot
    int64_t index;   // piece number in its sequence
    int64_t row0;    // first row of the sequence
    int64_t len;     // rows of the sequence
    int64_t first;   // first slot of the sequence
};

__device__ __forceinline__ int64_t clamp_offset(const Pieces& p, int64_t s)
{
    const int64_t v = p.offsets[s];
    return v < 0 ? 0 : (v > p.T ? p.T : v);
}

// Rows of sequence s and its first slot.
__device__ __forceinline__ Piece sequence_of(const Pieces& p, int64_t s)
{
    Piece r;
    r.seq = s;
    r.index = 0;
    if (!p.offsets) {
        r.row0 = s * p.T;
        r.len = p.T;
        r.first = s * p.per();
        return r;
    }
    r.row0 = clamp_offset(p, s);
    const int64_t hi = clamp_offset(p, s + 1);
    r.len = hi > r.row0 ? hi - r.row0 : 0;
    r.first = (r.row0 >> p.lg) + s;
    return r;
}

__device__ __forceinline__ Piece piece_of(const Pieces& p, int64_t slot)
{
    if (!p.offsets) {
        const int64_t per = p.per();
        int64_t s;
        if ((slot | per) >> 31)
            s = slot / per;
        else
            s = (uint32_t)slot / (uint32_t)per;
        Piece r = sequence_of(p, s);
        r.index = slot - s * per;
        return r;
    }
    // the last sequence whose first slot is not beyond this one
    int64_t lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if ((clamp_offset(p, mid) >> p.lg) + mid <= slot)
            lo = mid;
        else
            hi = mid;
    }
    Piece r = sequence_of(p, lo);
    r.index = slot - r.first;
    // idle: before the first sequence, or past this one's pieces (the empty
    // sequence's piece 0 exists)
    if (r.index < 0 || (r.index > 0 && (r.index << p.lg) >= r.len))
        r.seq = -1;
    return r;
}

// ---- rows ------------------------------------------------------------------
// V consecutive elements, one access (V > 1 when the caller has checked the
// alignment).
template <int V, typename T> __device__ __forceinline__ void store_row(T* p, const float* v)
{
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else {
        typedef T Vec __attribute__((ext_vector_type(V)));
        Vec x;
#pragma unroll
        for (int i = 0; i < V; ++i)
            x[i] = (T)v[i];
        *reinterpret_cast<Vec*>(p) = x;
    }
}

// The same elements unconverted: a load in flight holds half the registers.
template <typename T, int V> struct Raw {
    typedef T Type __attribute__((ext_vector_type(V)));
    static __device__ __forceinline__ Type load(const T* p) { return *reinterpret_cast<const Type*>(p); }
    static __device__ __forceinline__ Type zero() { Type z; for (int i = 0; i < V; ++i) z[i] = (T)0.f; return z; }
    static __device__ __forceinline__ void get(Type r, float* v)
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = (float)r[i];
    }
};
template <typename T> struct Raw<T, 1> {
    typedef T Type;
    static __device__ __forceinline__ Type load(const T* p) { return *p; }
    static __device__ __forceinline__ Type zero() { return (T)0.f; }
    static __device__ __forceinline__ void get(Type r, float* v) { v[0] = (float)r; }
};

// Every row of this matrix is whole, aligned vectors of V elements.
inline bool rows_aligned(const void* p, int64_t stride, int64_t width, int64_t elt, int V)
{
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)(V * elt) == 0 && stride % V == 0 && width % V == 0;
}

// ---- gate functions --------------------------------------------------------
// sigmoid on the exp2 and reciprocal units (each within 1 ulp).  Below about
// -88 the exponential is inf and the reciprocal 0, the right limit.
__device__ __forceinline__ float sigmoid_f(float x)
{
    return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * x));
}
// silu(x); -inf gives 0 * -inf = NaN in this form as in the formula's limit
// taken factor by factor.
__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }
// d silu / dx
__device__ __forceinline__ float silu_slope_f(float x)
{
    const float s = sigmoid_f(x);
    return s * (1.f + x * (1.f - s));
}

// ---- sums over lanes -------------------------------------------------------
template <int CTRL> __device__ __forceinline__ float dpp_move(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Lanes of the lower half (even rows) return the sum of a over the lane pair,
// the others that of b: one v_permlane*_swap and one add for two values.
__device__ __forceinline__ float pair_sum32(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
__device__ __forceinline__ float pair_sum16(float a, float b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Sum over aligned groups of W lanes (8 .. 64), in every lane: within a row of
// 16 by DPP (quads, then the mirrored half row and row: both partners hold
// their half's sum), across rows by a lane swap of the value with itself.
template <int W> __device__ __forceinline__ float lanes_sum(float v)
{
    v += dpp_quad_xor<1>(v);
    v += dpp_quad_xor<2>(v);
    v += dpp_move<0x141>(v);       // row_half_mirror
    if constexpr (W >= 16)
        v += dpp_move<0x140>(v);   // row_mirror
    if constexpr (W >= 32)
        v = pair_sum16(v, v);
    if constexpr (W >= 64)
        v = pair_sum32(v, v);
    return v;
}

}  // namespace gdr2
