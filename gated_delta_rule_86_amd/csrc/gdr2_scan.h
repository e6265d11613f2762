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

// NS fp32 per lane from / to a row of N states (zero past N).  One access per
// lane when whole lanes are in or out (N a multiple of NS; rows are then
// aligned to NS elements).
template <int NS>
__device__ __forceinline__ void load_states(const float* row, int s, int N, bool on, float (&h)[NS])
{
    typedef float Vec __attribute__((ext_vector_type(NS)));
    if (N % NS == 0) {
        Vec v;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            v[i] = 0.f;
        if (on && s * NS < N)
            v = *reinterpret_cast<const Vec*>(row + s * NS);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            h[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            h[i] = on && s * NS + i < N ? row[s * NS + i] : 0.f;
    }
}
template <int NS>
__device__ __forceinline__ void store_states(float* row, int s, int N, bool on, const float (&h)[NS])
{
    typedef float Vec __attribute__((ext_vector_type(NS)));
    if (N % NS == 0) {
        Vec v;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            v[i] = h[i];
        if (on && s * NS < N)
            *reinterpret_cast<Vec*>(row + s * NS) = v;
    } else {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (on && s * NS + i < N)
                row[s * NS + i] = h[i];
    }
}

// ---- loads ahead ----------------------------------------------------------
// A workgroup-uniform value the compiler cannot see to be one (it came through
// a vector load), kept in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ Piece uniform(const Piece& q)
{
    return {uniform(q.seq), uniform(q.index), uniform(q.row0), uniform(q.len), uniform(q.first)};
}

// Rows are read and written through buffer descriptors: the descriptor's
// base is the chunk's first row, its length ends behind the last row of the
// chunk that exists, and an access past the length reads 0 or writes nothing.
// So the tokens past a sequence cost no compare and no branch, and the lane
// offsets stay the same from chunk to chunk.
constexpr int kGroups = kScanChunk / 4;
constexpr uint32_t kNowhere = 0x80000000u;   // an offset past every length (32 rows, 2^24 elements apart, 4 bytes)

template <typename T> __device__ __forceinline__ auto chunk_buffer(const void* base, int64_t row, int64_t ld, int left)
{
    return __builtin_amdgcn_make_buffer_rsrc((void*)((T*)base + row * ld), (short)0, (int)(left * (int)ld * (int)sizeof(T)),
                                             0x00020000);
}
// A loaded element stays in a register of its own until it is used: as bf16
// the compiler would pack pairs, and wait for the loads to do so.
template <typename T, typename R> __device__ __forceinline__ uint32_t buffer_get(R rsrc, uint32_t off)
{
    if constexpr (sizeof(T) == 2)
        return __builtin_amdgcn_raw_buffer_load_b16(rsrc, off, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(rsrc, off, 0, 0);
}
template <typename T> __device__ __forceinline__ float raw_f32(uint32_t raw)
{
    return __builtin_bit_cast(float, sizeof(T) == 2 ? raw << 16 : raw);
}
template <typename T, typename R> __device__ __forceinline__ void buffer_put(R rsrc, uint32_t off, T v)
{
    if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), rsrc, off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rsrc, off, 0, 0);
}

// One row array of a chunk: this lane's elements are tokens 4 g + s.
template <typename T> struct TokenRows {
    uint32_t off[kGroups];
    __device__ __forceinline__ TokenRows(int64_t ld, int64_t c, int s, bool on)
    {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            off[g] = on ? (uint32_t)((4 * g + s) * (int)ld + (int)c) * (uint32_t)sizeof(T) : kNowhere;
    }
    __device__ __forceinline__ void load(const void* base, int64_t row, int64_t ld, int left, uint32_t (&raw)[kGroups]) const
    {
        const auto r = chunk_buffer<T>(base, row, ld, left);
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            raw[g] = buffer_get<T>(r, off[g]);
    }
};

// B or C of a chunk's tokens for group j, on their way to LDS as fp32
// [32][NP]: zero past the sequence and past N.
template <typename T, int NP> struct Staged {
    static constexpr int PER = kScanChunk * NP / 256;
    uint32_t off[PER], raw[PER];

    __device__ __forceinline__ Staged(int64_t ld, int64_t j, int N)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + 256 * i, r = e / NP, n = e % NP;
            off[i] = n < N ? (uint32_t)(r * (int)ld + (int)j * N + n) * (uint32_t)sizeof(T) : kNowhere;
        }
    }
    __device__ __forceinline__ void load(const void* base, int64_t row, int64_t ld, int left)
    {
        const auto r = chunk_buffer<T>(base, row, ld, left);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            raw[i] = buffer_get<T>(r, off[i]);
    }
    __device__ __forceinline__ void store(float (*dst)[NP]) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + 256 * i;
            dst[e / NP][e % NP] = raw_f32<T>(raw[i]);
        }
    }
};

// The steps of a chunk's tokens, all groups side by side (the eight chains of
// transcendentals fill each other's latencies); 0 past the sequence.
template <typename T>
__device__ __forceinline__ void chunk_steps(const uint32_t (&raw)[kGroups], float bias, int flags, int s, int left,
                                            float (&pre)[kGroups], float (&d)[kGroups])
{
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
        d[g] = pre[g] = raw_f32<T>(raw[g]) + bias;
    if (flags & GDR2_SCAN_SOFTPLUS) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            d[g] = softplus_f(pre[g]);
    }
    if (left < kScanChunk) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            d[g] = 4 * g + s < left ? d[g] : 0.f;
    }
}

// The states s NS .. of B and / or C for four tokens, in registers.  Read one
// group of tokens ahead of its use: a wave alone on its SIMD would otherwise
// stand still for the LDS at every token.
template <int NS> struct Quad {
    float v[4][NS];
    template <int NP> __device__ __forceinline__ void read(const float (*src)[NP], int tt, int s)
    {
        typedef float Vec __attribute__((ext_vector_type(NS < 4 ? NS : 4)));
        constexpr int W = NS < 4 ? NS : 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < NS; i += W) {
                const Vec x = *reinterpret_cast<const Vec*>(&src[tt + k][s * NS + i]);
#pragma unroll
                for (int e = 0; e < W; ++e)
                    v[k][i + e] = x[e];
            }
    }
};

}  // namespace gdr2
