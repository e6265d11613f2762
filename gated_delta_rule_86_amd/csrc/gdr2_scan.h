// gdr2_scan.h -- shared by the scan's forward and backward kernels: the lane
// layout, the per-token pieces and the segment plan.
//
// Lane layout.  A workgroup of 4 waves holds 64 channels of one group, 16 per
// wave; the four lanes of a quad hold one channel, lane s its states
// s*NS .. s*NS + NS-1 (NP = 4 NS >= N, the padding has B = C = 0).  Tokens are
// taken four at a time: lane s loads the rows' elements of token t + s, forms
// that token's step once, and hands it to its quad by a DPP broadcast; the
// four tokens' sums over the states come back the same way, one per lane.  So
// no load and no transcendental of a token is repeated over the quad, and the
// decay exponentials, the bulk of the work, are one per (token, channel, state).
// B and C of 32 tokens are staged in LDS in fp32 for the 64 channels.
#pragma once

#include "gdr2_layer.h"

namespace gdr2 {

constexpr int kScanChunk = GDR2_SCAN_CHUNK;   // tokens staged together, and between recorded states
constexpr int kScanLg = 5;
static_assert((1 << kScanLg) == kScanChunk, "chunk");
constexpr int kScanCols = 64;                 // channels of a workgroup

// softplus(x) = max(x, 0) + log(1 + e^-|x|), relatively accurate over the whole
// range (a step of 1e-5 scales the state's input as much as one of 0.1).
// u = e^-|x| is exp2 of the rounded product t = -|x| log2(e), corrected by what
// the rounding (of the product, by an fma, and of the constant) left out;
// log(1 + u) is log(w) u / (w - 1) with w = fl(1 + u), where the rounding of w
// cancels between log(w) and w - 1.
__device__ __forceinline__ float softplus_f(float x)
{
    constexpr float kLog2eLow = 1.92596299e-8f;   // log2(e) - fl(log2(e))
    const float ax = fabsf(x), t = -kLog2e * ax;
    const float rest = fmaf(-kLog2e, ax, -t) - kLog2eLow * ax;
    const float e = fast_exp2(t), u = fmaf(e, rest * 0.693147181f, e);
    const float w = 1.f + u;
    const float l = w == 1.f ? u : __logf(w) * (u * __builtin_amdgcn_rcpf(w - 1.f));
    return fmaxf(x, 0.f) + l;
}

// Lane k of every quad broadcast to its quad.
template <int K> __device__ __forceinline__ float quad_bcast(float v)
{
    constexpr int ctrl = K * 0x55;   // quad_perm [K, K, K, K]
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xF, 0xF, true));
}
__device__ __forceinline__ float quad_bcast_k(float v, int k)   // k a compile-time constant after unrolling
{
    return k == 0 ? quad_bcast<0>(v) : k == 1 ? quad_bcast<1>(v) : k == 2 ? quad_bcast<2>(v) : quad_bcast<3>(v);
}

// p[k] of the four lanes of a quad: lane s returns the sum of p[s].
__device__ __forceinline__ float quad_sum_transposed(const float (&p)[4], int s)
{
    const bool b0 = s & 1, b1 = s & 2;
    const float q0 = (b0 ? p[1] : p[0]) + dpp_quad_xor<1>(b0 ? p[0] : p[1]);
    const float q1 = (b0 ? p[3] : p[2]) + dpp_quad_xor<1>(b0 ? p[2] : p[3]);
    return (b1 ? q1 : q0) + dpp_quad_xor<2>(b1 ? q0 : q1);
}

// Segments of a scan: L = 2^lg tokens each.
struct ScanPlan {
    Pieces seg;
    int64_t ncb;      // channel blocks: G * ceil(C / G / 64)
    int64_t cb_per;   // per group
    bool split;       // sequences may have more than one segment
};
ScanPlan scan_plan(const gdr2_scan_args& a, bool backward);

// This lane's place.
struct ScanLane {
    int64_t c;     // channel, or C when the lane has none
    int64_t j;     // group
    int s;         // lane of the quad
    bool on;
};
__device__ __forceinline__ ScanLane scan_lane(const gdr2_scan_args& a, uint32_t cb, uint32_t cb_per)
{
    ScanLane l;
    const uint32_t j = cb / cb_per;
    const int64_t cg = a.C / a.G;
    const int64_t in = (int64_t)(cb - j * cb_per) * kScanCols + (threadIdx.x >> 2);
    l.j = j;
    l.s = threadIdx.x & 3;
    l.on = in < cg;
    l.c = j * cg + (l.on ? in : 0);
    return l;
}

// NS fp32 per lane from / to a row of N states (zero past N).
template <int NS>
__device__ __forceinline__ void load_states(const float* row, int s, int64_t N, bool on, float (&h)[NS])
{
#pragma unroll
    for (int i = 0; i < NS; ++i)
        h[i] = on && s * NS + i < N ? row[s * NS + i] : 0.f;
}
template <int NS>
__device__ __forceinline__ void store_states(float* row, int s, int64_t N, bool on, const float (&h)[NS])
{
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (on && s * NS + i < N)
            row[s * NS + i] = h[i];
}

// B and / or C of the tokens t .. t + 31 of group j into LDS, fp32 [32][NP],
// zero past the sequence and past N.
template <typename T, int NP>
__device__ __forceinline__ void stage_rows(const void* base, int64_t ld, int64_t row0, int64_t t, int64_t len, int64_t j,
                                           int64_t N, float (*dst)[NP])
{
    for (int e = threadIdx.x; e < kScanChunk * NP; e += 256) {
        const int r = e / NP, n = e % NP;
        float v = 0.f;
        if (t + r < len && n < N)
            v = to_f32(((const T*)base)[(row0 + t + r) * ld + j * N + n]);
        dst[r][n] = v;
    }
}

}  // namespace gdr2
