// gdr2_scan.h -- shared by the scan's forward and backward kernels: the lane
// layout, the per-token pieces and the segment plan.
//
// Two layouts share the work of a chunk of 32 tokens x 64 channels of a group:
//
//   rows     thread (token, V adjacent channels): 2048 elements over 64 LPC
//            threads.  Row arrays move in whole 128-byte
//            lines, each requested once per workgroup, and everything that is
//            per (token, channel) is done here: the steps, the gate, stores.
//   states   LPC adjacent lanes hold one channel, lane s its states s NS ..
//            s NS + NS - 1 (NP = LPC NS >= N; the padding has B = C = 0), and
//            walk the tokens one after the other.  Everything that is per
//            (token, channel, state) is done here: the decay exponentials, the
//            recurrence, the product with C.
//
// The forward kernel has waves of its own for each; in the others the same waves
// do both in turn.  LDS carries (d, d x) from rows to states and the sums over n back; B and C
// are staged there in fp32 for the 64 channels.
#pragma once

#include "gdr2_layer.h"

namespace gdr2 {

constexpr int kScanChunk = GDR2_SCAN_CHUNK;   // tokens staged together, and between recorded states
constexpr int kScanLg = 5;
static_assert((1 << kScanLg) == kScanChunk, "chunk");
constexpr int kScanCols = 64;                 // channels of a workgroup

// softplus(x) = max(x, 0) + log(1 + e^-|x|), relatively accurate over the whole
// range (a step of 1e-5 scales the state's input as much as one of 0.1): within
// 3e-7 on [-60, 10], for rows of either type, whose states are fp32.
// u = e^-|x| is exp2 of the rounded product t = -|x| log2(e); e = -|x| - t ln 2,
// by fmas, is what the exponent is off by, and u e what u is (without it 3.5e-6;
// it costs 1 to 3 % of a bf16 call in segments, nothing of one in one pass).
// log(1 + u) is log(w) + (u - (w - 1)) with w = fl(1 + u): what w rounded away,
// at most 2^-24, is added back (over w by the derivative; leaving that factor
// out costs 2^-24 u).
// |x| goes in as at most 128, where u is 0: a larger one (a step masked with
// -inf or the lowest value) would make t, and then the correction, infinite.
// (The minimum of a NaN is NaN.)
__device__ __forceinline__ float softplus_f(float x)
{
    constexpr float kLn2 = 0.693147181f, kLn2Low = -1.90465432e-9f;   // ln 2 - fl(ln 2)
    const float ax = __builtin_elementwise_minimum(fabsf(x), 128.f), t = -kLog2e * ax, u = fast_exp2(t);
    const float e = fmaf(-t, kLn2Low, fmaf(-t, kLn2, -ax)), w = 1.f + u;
    return fmaxf(x, 0.f) + fmaf(kLn2, __builtin_amdgcn_logf(w), fmaf(u, e, u - (w - 1.f)));
}

// p[k] of the LPC lanes of a channel: lane s returns the sum of p[s].  Each
// round adds half of the values to the partner that keeps the other half.
__device__ __forceinline__ float sum_transposed(const float (&p)[4], int s)
{
    const bool b0 = s & 1, b1 = s & 2;
    const float q0 = (b0 ? p[1] : p[0]) + dpp_quad_xor<1>(b0 ? p[0] : p[1]);
    const float q1 = (b0 ? p[3] : p[2]) + dpp_quad_xor<1>(b0 ? p[2] : p[3]);
    return (b1 ? q1 : q0) + dpp_quad_xor<2>(b1 ? q0 : q1);
}
__device__ __forceinline__ float sum_transposed(const float (&p)[8], int s)
{
    // the partner of the first round is lane 7 - s of the eight
    const bool b2 = s & 4;
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        q[k] = (b2 ? p[4 + k] : p[k]) + dpp_move<0x141>(b2 ? p[k] : p[4 + k]);
    return sum_transposed(q, s);
}

// Segments of a scan: L = 2^lg tokens each.
struct ScanPlan {
    Pieces seg;
    int64_t ncb;      // channel blocks: G * ceil(C / G / 64)
    int64_t cb_per;   // per group
    bool split;       // sequences may have more than one segment
};
ScanPlan scan_plan(const gdr2_scan_args& a, bool backward);
constexpr int kFoldAhead = 8;     // segments whose values the folds load together

// This lane's place in the states layout.
struct ScanLane {
    int64_t c;     // channel (the block's first when the lane has none)
    int s;         // lane of the channel
    bool on;
};
// The workgroup's channels: c0 .. c0 + n - 1 of group j.
struct ScanBlock {
    int64_t j, c0;
    int n;
};
__device__ __forceinline__ ScanBlock scan_block(const gdr2_scan_args& a, uint32_t cb, uint32_t cb_per)
{
    ScanBlock b;
    const uint32_t j = cb / cb_per;
    const int64_t cg = a.C / a.G, in = (int64_t)(cb - j * cb_per) * kScanCols;
    b.j = j;
    b.c0 = j * cg + in;
    b.n = (int)min(cg - in, (int64_t)kScanCols);
    return b;
}
template <int LPC> __device__ __forceinline__ ScanLane scan_lane(const ScanBlock& b)
{
    const int i = threadIdx.x % (64 * LPC) / LPC;
    return {b.c0 + (i < b.n ? i : 0), (int)(threadIdx.x % LPC), i < b.n};
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

// Waits for this wave's LDS accesses, then for the workgroup.  (__syncthreads()
// would also wait for loads and stores in flight, which are left to run across
// chunks.)
__device__ __forceinline__ void lds_barrier() { __asm__ __volatile__("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

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
constexpr uint32_t kNowhere = 0x80000000u;   // an offset past every length (32 rows, 2^24 elements apart, 4 bytes)

// A row array walked chunk by chunk, in scalar registers: the address of a
// chunk's first row and the bytes of one row.
struct RowWalk {
    const char* base;
    uint32_t row_bytes;

    template <typename T> static __device__ __forceinline__ RowWalk at(const void* p, int64_t row, int64_t ld)
    {
        return {(const char*)((const T*)p + row * ld), (uint32_t)ld * (uint32_t)sizeof(T)};
    }
    __device__ __forceinline__ void advance(int rows) { base += (int64_t)rows * (int32_t)row_bytes; }
    // `left` rows from the base on
    __device__ __forceinline__ auto buffer(int left) const
    {
        return __builtin_amdgcn_make_buffer_rsrc((void*)uniform((int64_t)base), (short)0,
                                                 __builtin_amdgcn_readfirstlane((int)(left * row_bytes)), 0x00020000);
    }
};
template <typename T> __device__ __forceinline__ float raw_f32(uint32_t raw)
{
    return __builtin_bit_cast(float, sizeof(T) == 2 ? raw << 16 : raw);
}
template <typename T, typename R> __device__ __forceinline__ uint32_t buffer_get(R rsrc, uint32_t off)
{
    if constexpr (sizeof(T) == 2)
        return __builtin_amdgcn_raw_buffer_load_b16(rsrc, off, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(rsrc, off, 0, 0);
}

// The rows layout of one array: V channels of one token of every chunk.
// WIDE: rows and blocks are aligned to V elements, which then move together;
// otherwise one by one.  Loaded elements stay as they are until they are used.
template <typename T, int V, bool WIDE> struct RowVec {
    static constexpr int W = V * (int)sizeof(T) / 4;          // registers of a packed vector
    static constexpr int REGS = WIDE ? W : V;
    uint32_t off;
    int n;             // channels of the vector that exist
    uint32_t raw[REGS];

    __device__ __forceinline__ RowVec(int64_t ld, const ScanBlock& b)
    {
        const int token = threadIdx.x / (kScanCols / V) % kScanChunk, ch = threadIdx.x % (kScanCols / V) * V;
        n = min(V, max(0, b.n - ch));
        off = n > 0 ? (uint32_t)(token * (int)ld + (int)b.c0 + ch) * (uint32_t)sizeof(T) : kNowhere;
    }
    __device__ __forceinline__ uint32_t at(int v) const { return v < n ? off + v * (uint32_t)sizeof(T) : kNowhere; }

    __device__ __forceinline__ void load(const RowWalk& walk, int left)
    {
        const auto r = walk.buffer(left);
        if constexpr (WIDE) {
#pragma unroll
            for (int w = 0; w < W; w += 4) {
                typedef uint32_t U4 __attribute__((ext_vector_type(4)));
                typedef uint32_t U2 __attribute__((ext_vector_type(2)));
                if constexpr (W == 2) {
                    const U2 x = __builtin_bit_cast(U2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
                    raw[0] = x[0];
                    raw[1] = x[1];
                } else {
                    const U4 x = __builtin_bit_cast(U4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * w, 0, 0));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        raw[w + i] = x[i];
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                raw[v] = buffer_get<T>(r, at(v));
        }
    }
    __device__ __forceinline__ float get(int v) const
    {
        if constexpr (WIDE && sizeof(T) == 2)
            return __builtin_bit_cast(float, v & 1 ? raw[v / 2] & 0xffff0000u : raw[v / 2] << 16);
        else
            return raw_f32<T>(raw[v]);
    }
    __device__ __forceinline__ void store(const RowWalk& walk, int left, const float (&y)[V]) const
    {
        const auto r = walk.buffer(left);
        if constexpr (WIDE) {
            typedef T VecT __attribute__((ext_vector_type(V)));
            VecT o;
#pragma unroll
            for (int v = 0; v < V; ++v)
                o[v] = (T)y[v];
            typedef uint32_t UW __attribute__((ext_vector_type(W)));
            typedef uint32_t U4 __attribute__((ext_vector_type(4)));
            const UW x = __builtin_bit_cast(UW, o);
            if constexpr (W == 2) {
                __builtin_amdgcn_raw_buffer_store_b64(x, r, off, 0, 0);
            } else {
#pragma unroll
                for (int w = 0; w < W; w += 4)
                    __builtin_amdgcn_raw_buffer_store_b128(U4{x[w], x[w + 1], x[w + 2], x[w + 3]}, r, off + 4 * w, 0, 0);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if constexpr (sizeof(T) == 2)
                    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)y[v]), r, at(v), 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, y[v]), r, at(v), 0, 0);
            }
        }
    }
};

// B or C of a chunk's tokens for group j, on their way to LDS as fp32
// [32][NP]: zero past the sequence and past N.
template <typename T, int NP, int NT> struct Staged {
    static constexpr int PER = kScanChunk * NP / NT;
    uint32_t off[PER], raw[PER];

    __device__ __forceinline__ Staged(int64_t ld, int64_t j, int N)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x % NT + NT * i, r = e / NP, n = e % NP;
            off[i] = n < N ? (uint32_t)(r * (int)ld + (int)j * N + n) * (uint32_t)sizeof(T) : kNowhere;
        }
    }
    __device__ __forceinline__ void load(const RowWalk& walk, int left)
    {
        const auto r = walk.buffer(left);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            raw[i] = buffer_get<T>(r, off[i]);
    }
    __device__ __forceinline__ void store(float (*dst)[NP]) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x % NT + NT * i;
            dst[e / NP][e % NP] = raw_f32<T>(raw[i]);
        }
    }
};

// Whether every row array and block of a call moves V elements at a time.
inline bool scan_wide(const gdr2_scan_args& a, int V)
{
    const int64_t e = a.dtype == GDR2_BF16 ? 2 : 4, cg = a.C / a.G;
    auto ok = [&](const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % (V * e) == 0 && ld % V == 0); };
    return cg % V == 0 && ok(a.x, a.x_stride) && ok(a.dt, a.dt_stride) && ok(a.z, a.z_stride);
}

// What one token needs in the states layout, read from LDS LPC tokens ahead of
// its use: with few waves on a SIMD nothing else hides the LDS.  (d, d x) of
// two tokens lie together there, [token / 2][channel][d, dx, d', dx'], so that
// one read serves two.
constexpr int kStepLd = 4 * kScanCols;

// Where a channel's 16 bytes of a token lie in LDS.  A thread of the rows
// layout writes 8 (or 4) channels in turn; in channel order the lanes of a
// wave would be 128 bytes apart, all on the same banks.
__device__ __forceinline__ int step_place(int channel) { return channel ^ ((channel >> 3) & 7); }

template <int NS> __device__ __forceinline__ void read_states(const float* p, float (&v)[NS])
{
    typedef float Vec __attribute__((ext_vector_type(NS)));
    const Vec x = *reinterpret_cast<const Vec*>(p);
#pragma unroll
    for (int i = 0; i < NS; ++i)
        v[i] = x[i];
}

// This thread's channels (rows layout) of a per-channel parameter; 0 without.
template <int V> __device__ __forceinline__ void channel_params(const float* p, const ScanBlock& b, float (&out)[V])
{
    const int ch = threadIdx.x % (kScanCols / V) * V;
#pragma unroll
    for (int v = 0; v < V; ++v)
        out[v] = p && ch + v < b.n ? p[b.c0 + ch + v] : 0.f;
}

// A and log2(e) A, kept finite: the tokens past a sequence have d = 0, and d
// times an infinite A would be NaN in the state they are to leave as it is.
// (A NaN stays one.)
__device__ __forceinline__ float finite(float v)
{
    v = v < -__FLT_MAX__ ? -__FLT_MAX__ : v;
    return v > __FLT_MAX__ ? __FLT_MAX__ : v;
}
__device__ __forceinline__ float exponent_scale(float A) { return finite(A * kLog2e); }

// 2^t h + e, t a whole segment's exponent.  Where 2^t nears the ends of the
// format it would be inf or 0 while the state, before and after, is neither
// (and inf times a zero state NaN): there it is applied in two halves.  At
// +-254 these are finite, and any normal state goes out of range or to 0 with
// them.  (A NaN t stays one.)
__device__ __forceinline__ float segment_decay(float t, float h, float e)
{
    const float c = __builtin_elementwise_maximum(__builtin_elementwise_minimum(t, 254.f), -254.f);
    const float half = fabsf(c) > 120.f ? 0.5f * c : 0.f;
    return fmaf(fast_exp2(c - half), fast_exp2(half) * h, e);
}

// The step from its raw value.  softplus is formed either way: behind a branch
// per element it would split the block it is scheduled in.
__device__ __forceinline__ float step_of(float raw, bool softplus)
{
    float soft = softplus_f(raw);
    asm volatile("" : "+v"(soft));
    return softplus ? soft : raw;
}

}  // namespace gdr2
