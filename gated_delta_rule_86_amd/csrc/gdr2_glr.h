// gdr2_glr.h -- shared by the gated linear recurrence's forward and backward
// kernels: the lane layout, the per-token terms and the segment plan.
//
// The recurrence h_t = a_t h_{t-1} + b_t is linear in the state, so a run of
// tokens maps the state before it to the one after it by h -> P h + L (P the
// product of its decays, L its end state from zero), and runs join:
// (P2, L2) after (P1, L1) is (P2 P1, P2 L1 + L2).  A workgroup owns LR V
// channels and walks a sequence in tiles:
//
//   sub-chunk  16 tokens of V adjacent channels of one lane.  LR lanes lie
//              along the channels, so that a wave moves whole 128-byte lines (LR V
//              elements a row; with halves of them 8x4096x2048 takes 156 us, not
//              112), and 64 / LR sub-chunks side by side in time;
//   tile       the sub-chunks of the workgroup's waves, kSubs of them.
//
// Each lane forms its decays and inputs once, in registers, and its (P, L);
// through LDS it then finds the state its sub-chunk starts from, and walks its
// tokens.  So every element is read once, its transcendentals are evaluated once, and
// the state's chain is one multiply-add per sub-chunk, not per token.
//
// Where sequences are too few to fill the chip so, every tile is a workgroup of
// its own (a chain): it hands its (P, L) on through device memory, finds the
// state it starts from by the (P, L) of the tiles before it, back to one whose
// state is there, and hands on the state behind it.  Elements are still read once.
#pragma once

#include "gdr2_block.h"
#include "gdr2_scan.h"

namespace gdr2 {

constexpr int kGlrChunk = GDR2_GLR_CHUNK;     // tokens of a sub-chunk, and between recorded states
// NW: waves of a workgroup.
template <int LR, int NW> struct GlrTile {
    static constexpr int kGroups = 64 / LR;                     // sub-chunks of a wave
    static constexpr int kSubs = NW * kGroups;           // of a tile
    static constexpr int kWaveTokens = kGroups * kGlrChunk;
    static constexpr int kTokens = kSubs * kGlrChunk;
};

// What tiles hand on, in device memory.  A map is (P, L), a state (h, 1); each is
// one 64-bit word, so that it is there whole or not at all.
struct GlrChain {
    uint32_t* tickets;     // one for each channel block, 128 bytes apart
    uint64_t* maps;        // [slots][C]
    uint64_t* states;      // [slots][C]
};
constexpr int kTicketWords = 32;
constexpr uint32_t kNoMap = 0xbf800000u;     // P = -1, which no product of exponentials is

// How a call's workgroups are laid out: pieces of whole sequences (or, chained,
// of one tile), and channel blocks.
struct GlrPlan {
    Pieces seg;
    int64_t blocks;    // of channels
    bool chained;
    int64_t chain_words() const { return chained ? blocks * (kTicketWords / 2) + 2 * seg.slots() * C : 0; }
    int64_t C;
    GlrChain chain(void* workspace) const
    {
        uint64_t* w = (uint64_t*)workspace;
        uint64_t* maps = w + blocks * (kTicketWords / 2);
        return {(uint32_t*)w, maps, maps + seg.slots() * C};
    }
};
// Waves of a workgroup.  One pass: two on each SIMD.  Chained tiles: as many for
// the forward, fewer for the gradients, which take more registers: three
// workgroups a compute unit (4x4096x2048 from 8 bits: eight waves 143 us, four 126).
constexpr int kGlrWaves = 8, kChainedBackwardWaves = 4;
GlrPlan glr_plan(const gdr2_glr_args& a, int V, bool backward);
// Empties a chain.
hipError_t launch_glr_chain_reset(const GlrPlan& plan, void* workspace, hipStream_t stream);

// Whether a lane holds two channels: bf16 where every row array is aligned to
// pairs.  (One of fp32 is as wide, and 64 lanes of them 256 bytes.)
inline bool glr_pairs(const gdr2_glr_args& a)
{
    auto ok = [&](const void* p, int64_t ld) { return !p || (reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0); };
    return a.dtype == GDR2_BF16 && a.C % 2 == 0 && ok(a.x, a.x_stride) && ok(a.r, a.r_stride) && ok(a.i, a.i_stride);
}

// ---- rows of a sub-chunk ---------------------------------------------------
// A sub-chunk's rows are addressed by one offset that goes on by a row per
// token: formed from the token's number they would be invariants of the tiles'
// loop, and fill the registers.  Tokens past the sequence lie past the
// descriptor's end: they read 0 and write nothing.
struct RowOffset {
    uint32_t at, row_bytes;
    __device__ __forceinline__ uint32_t next()
    {
        const uint32_t v = at;
        at += row_bytes;
        asm("" : "+v"(at));
        return v;
    }
};

// Cache policy of loads: read once (nt) where rows are whole lines, forwards
// 8x4096x2048 127 -> 112 us.  Where they are not, two workgroups share the lines
// at their blocks' ends, and the cache should keep them: forwards fp32
// 5x3001x1003 67 -> 62 us, bf16 49 -> 44, 15x3001x1002 90 -> 83, with 8-bit rows 8x3001x2050 220 -> 197.
// (Gradients have one policy: with the other fp32 16x3001x1003 363 -> 304, but
// 32x1000x500 87 -> 101, chained 5x3001x1003 121 -> 131.  What divides them is open.)
constexpr int kOnce = 2, kKeep = 0;
inline bool glr_whole_lines(const gdr2_glr_args& a)
{
    const int64_t e = a.dtype == GDR2_BF16 ? 2 : 4;
    auto ok = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 128 == 0 && ld * e % 128 == 0; };
    return ok(a.x, a.x_stride) && ok(a.r, a.r_stride) && ok(a.i, a.i_stride);
}

// The V elements of every token as they lie in memory, a register each.
template <typename T, int V> struct SubRows {
    static_assert(V * sizeof(T) <= 4, "one register");
    uint32_t raw[kGlrChunk];

    template <int POLICY = kOnce, typename R> __device__ __forceinline__ void load(int k, R rsrc, RowOffset& at)
    {
        if constexpr (V * sizeof(T) == 2)
            raw[k] = __builtin_amdgcn_raw_buffer_load_b16(rsrc, at.next(), 0, POLICY);
        else
            raw[k] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at.next(), 0, POLICY);
    }
    __device__ __forceinline__ float get(int k, int v) const
    {
        if constexpr (sizeof(T) == 4)
            return __builtin_bit_cast(float, raw[k]);
        else
            return __builtin_bit_cast(float, v ? raw[k] & 0xffff0000u : raw[k] << 16);
    }
    // Tokens past the sequence (from `left` on) as masked ones: a = 1, and the
    // state passes them.
    __device__ __forceinline__ void mask(int left)
    {
#pragma unroll
        for (int k = 0; k < kGlrChunk; ++k)
            raw[k] = k < left ? raw[k] : sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    }
};

template <typename T, int V, typename R> __device__ __forceinline__ void store_token(R rsrc, uint32_t at, const float (&v)[V])
{
    if constexpr (V == 2) {
        typedef T Vec __attribute__((ext_vector_type(2)));
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (Vec){(T)v[0], (T)v[1]}), rsrc, at, 0, 0);
    } else if constexpr (sizeof(T) == 4) {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[0]), rsrc, at, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)v[0]), rsrc, at, 0, 0);
    }
}

// One array's rows in memory, from the wave's first row of a tile on.
struct WaveRows {
    const char* base;
    uint32_t row_bytes;
    template <typename T> static __device__ __forceinline__ WaveRows at(const void* p, int64_t row, int64_t ld)
    {
        return {(const char*)((const T*)p + row * ld), (uint32_t)ld * (uint32_t)sizeof(T)};
    }
    // `left` rows from `row` rows behind the base
    __device__ __forceinline__ auto buffer(int64_t row, int left) const
    {
        return __builtin_amdgcn_make_buffer_rsrc((void*)uniform((int64_t)(base + row * (int64_t)row_bytes)), (short)0,
                                                 __builtin_amdgcn_readfirstlane((int)((uint32_t)left * row_bytes)), 0x00020000);
    }
};

// ---- the terms of a token --------------------------------------------------
// q = sqrt(1 - a^2) = sqrt(-expm1(w)), w = 2 A s(r) = 2 ln 2 t with t = A2 s(r).
// Near w = 0 the difference cancels, so -expm1(w) = -(w + w^2/2 + .. + w^5/120)
// there, a polynomial in t: at |w| <= 1/8 the first term left out is w^5/720 <
// 5e-8 of the value, and beyond it 1 - a^2 >= 0.117 has lost three bits at most.
__device__ __forceinline__ float glr_root(float t, float a)
{
    constexpr float c = 1.386294361f;
    float p = fmaf(t, -c * c * c * c * c / 120.f, -c * c * c * c / 24.f);
    p = fmaf(p, t, -c * c * c / 6.f);
    p = fmaf(p, t, -c * c / 2.f);
    p = fmaf(p, t, -c) * t;
    return __builtin_amdgcn_sqrtf(__builtin_unpredictable(t > -0.125f / c) ? p : fmaf(-a, a, 1.f));
}

// 0 for a masked token (q == 0), whose x and i may be anything, NaN among them.
// (Unpredictable, that is a select: a branch per element would split the block
// it is scheduled in.)
__device__ __forceinline__ float unless_masked(float q, float v) { return __builtin_unpredictable(q == 0.f) ? 0.f : v; }

// This workgroup's slot and channel block.
struct GlrWork {
    int64_t slot, block;
};
// Workgroups go to the eight XCDs in turn; numbered so, an XCD owns a range of
// neighbouring channel blocks, and its cache sees whole rows: every
// eighth block of 128 bytes would fall into a few of its channels.
__device__ __forceinline__ uint32_t xcd_ranges(uint32_t at, uint32_t count)
{
    const uint32_t n = count / 8, rest = count % 8, xcd = at % 8;
    return xcd * n + (xcd < rest ? xcd : rest) + at / 8;
}
__device__ __forceinline__ GlrWork one_pass_work(const GlrPlan& plan)
{
    const uint32_t id = xcd_ranges(blockIdx.x, gridDim.x);
    const int64_t slot = id / plan.blocks;
    return {slot, id - slot * plan.blocks};
}
// Chained: tiles are taken in the order of their tickets, so that the tiles one
// waits for are taken by workgroups that run already, and wait only for such
// themselves.
__device__ __forceinline__ GlrWork chained_work(const GlrPlan& plan, const GlrChain& chain, bool reverse)
{
    __shared__ uint32_t s_ticket;
    const int64_t block = xcd_ranges(blockIdx.x % (uint32_t)plan.blocks, (uint32_t)plan.blocks);
    if (threadIdx.x == 0)
        s_ticket = atomicAdd(chain.tickets + block * kTicketWords, 1u);
    __syncthreads();
    const int64_t ticket = uniform((int64_t)s_ticket);
    return {reverse ? plan.seg.slots() - 1 - ticket : ticket, block};
}

__device__ __forceinline__ void hand_on(uint64_t* to, uint32_t low, uint32_t high)
{
    __hip_atomic_store(to, (uint64_t)high << 32 | low, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t handed(const uint64_t* from)
{
    return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The state of channel c behind the `count` > 0 tiles before `slot` (in steps of
// `step`): the nearest one that is there, and the maps from it on.  Maps are
// applied one by one, as the tile whose state it is applied those before it, so
// the result does not depend on which state was found.  Every slot's state is
// handed on in the end, whatever the offsets say, so the wait ends.
__device__ __forceinline__ float state_behind(const GlrChain& chain, int64_t slot, int step, int64_t count, int64_t C, uint32_t c)
{
    constexpr int kBack = 4;      // tiles looked at together: their words are a round trip away
                                  // (gradients 4x4096x2048: 2 and 4 alike, 8 fills the registers, 122 -> 149 us)
    for (;;) {
        uint64_t maps[kBack], states[kBack];
#pragma unroll
        for (int u = 0; u < kBack; ++u) {
            maps[u] = kNoMap;
            states[u] = 0;
            if (u < count) {
                const int64_t row = (slot + (int64_t)step * (u + 1)) * C;     // the same for all lanes
                maps[u] = handed(chain.maps + row + c);
                states[u] = handed(chain.states + row + c);
            }
        }
        int found = kBack;
        bool open = true;
#pragma unroll
        for (int u = 0; u < kBack; ++u) {
            const bool state = (uint32_t)(states[u] >> 32) != 0;
            if (open && state)
                found = u;
            open = open && !state && (uint32_t)maps[u] != kNoMap;
        }
        if (found < kBack) {
            float h = 0.f;
#pragma unroll
            for (int u = kBack - 1; u >= 0; --u) {
                const float P = __builtin_bit_cast(float, (uint32_t)maps[u]), L = __builtin_bit_cast(float, (uint32_t)(maps[u] >> 32));
                if (u == found)
                    h = __builtin_bit_cast(float, (uint32_t)states[u]);
                else if (u < found)
                    h = fmaf(P, h, L);
            }
            return h;
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

// By the first wave, a lane a channel: the tile's map from its N sub-chunks', in
// the order FIRST, FIRST + STEP, .., then the state it starts from, then the one behind it.
// `begin`: the state where the tile is its sequence's first in this direction.
template <int V, int LR, int N, int STEP>
__device__ __forceinline__ float chain_state(const GlrChain& chain, const float (*s_span)[LR][2 * V], int64_t slot, int64_t before,
                                             int64_t C, int64_t c, const float* begin)
{
    const int li = threadIdx.x / V, v = threadIdx.x % V;
    float P = 1.f, L = 0.f;
#pragma unroll 4
    for (int k = 0; k < N; ++k) {
        const int j = STEP > 0 ? k : N - 1 - k;
        const float p = s_span[j][li][2 * v], l = s_span[j][li][2 * v + 1];
        L = fmaf(p, L, l);
        P *= p;
    }
    if (c >= C)
        return 0.f;
    hand_on(chain.maps + slot * C + c, __builtin_bit_cast(uint32_t, P), __builtin_bit_cast(uint32_t, L));
    const float h = before > 0 ? state_behind(chain, slot, -STEP, before, C, (uint32_t)c) : begin ? begin[c] : 0.f;
    hand_on(chain.states + slot * C + c, __builtin_bit_cast(uint32_t, fmaf(P, h, L)), 1u);
    return h;
}
// What an idle slot hands on: nothing changes.
__device__ __forceinline__ void chain_idle(const GlrChain& chain, int64_t slot, int64_t C, int64_t c)
{
    if (threadIdx.x < 64 && c < C) {
        hand_on(chain.maps + slot * C + c, __builtin_bit_cast(uint32_t, 1.f), 0u);
        hand_on(chain.states + slot * C + c, 0u, 1u);
    }
}

// Where this lane's channels and sub-chunk lie.
template <int V, int LR> struct GlrLane {
    int li, sub, wave;
    int64_t c;
    bool on;
    __device__ __forceinline__ GlrLane(int64_t C, int64_t block)
    {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        li = lane % LR;
        sub = wave * (64 / LR) + lane / LR;
        c = block * (LR * V) + li * V;
        on = c < C;
    }
    // offset in an array's rows from the wave's first one
    template <typename T> __device__ __forceinline__ uint32_t offset(uint32_t row_bytes) const
    {
        return on ? (uint32_t)((threadIdx.x & 63) / LR) * kGlrChunk * row_bytes + (uint32_t)c * (uint32_t)sizeof(T) : kNowhere;
    }
    // the same for the scale of the block its channels lie in, which the lanes
    // past the row's end share with those before it
    __device__ __forceinline__ uint32_t scale_offset(uint32_t row_bytes, int64_t C) const
    {
        const int64_t at = c / kRows8;
        return at < scale_count(C) ? (uint32_t)((threadIdx.x & 63) / LR) * kGlrChunk * row_bytes + (uint32_t)at : kNowhere;
    }
};

// This workgroup's segment: `n` tokens from token `t0` of the sequence on.
struct Segment {
    Piece q;
    int64_t t0, n;
};
__device__ __forceinline__ Segment segment_of(const GlrPlan& plan, int64_t slot)
{
    Segment s;
    s.q = uniform(piece_of(plan.seg, slot));
    s.t0 = s.q.index << plan.seg.lg;
    const int64_t rest = s.q.len - s.t0, L = (int64_t)1 << plan.seg.lg;
    s.n = rest < L ? rest : L;
    return s;
}

// Rows of 16 tokens before a sequence's first one in h_chunks.
__device__ __forceinline__ int64_t chunk_row(const gdr2_glr_args& a, const Piece& q)
{
    return a.offsets ? q.row0 / kGlrChunk + q.seq : q.seq * ((a.T + kGlrChunk - 1) / kGlrChunk);
}

template <int V> __device__ __forceinline__ void load_channels(const float* p, float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = p[i];
}
template <int V> __device__ __forceinline__ void store_channels(float* p, const float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i)
        p[i] = v[i];
}

}  // namespace gdr2
