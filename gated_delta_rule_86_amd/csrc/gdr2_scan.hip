// gdr2_scan.hip -- the selective state space scan, forwards: prompts (one
// pass, or segments of long sequences in parallel) and single tokens.
//
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   v_t = C_t . h_t + skip x_t,
//   y_t = v_t silu(z_t)
//
// Per (token, channel, state): one multiply for the exponent, one exp2, and
// three multiply-adds.  At 16 states that arithmetic, not the 8 bytes a channel
// moves per token, bounds a prompt: 8 x 4096 x 2048 channels, gated, in bf16 take
// 255 us, of which the exponentials, multiplies and adds are 178 us at the issue
// rate measured for them (4.3 cycles a wave, 8.9 for exp2) and the 540 MB 106 us
// at the rate of a large copy.
//
// Segments: h is linear in its start, so over a segment h_end = P h_start + E
// with P = exp(A sum d) and E the end state from zero.  A span pass forms
// (sum d, E) of every segment but a sequence's last, a fold chains the
// segments' start states, and the main pass runs them all at once.
#include <algorithm>

#include "gdr2_scan.h"

namespace gdr2 {

namespace {

// (d, d x) of one channel of a thread's row vector into LDS; 0 past the
// sequence, where the token then leaves the state as it is.
__device__ __forceinline__ void step_to_lds(float dt, float x, float bias, bool softplus, bool in, float* at)
{
    typedef float Two __attribute__((ext_vector_type(2)));
    float d = step_of(dt + bias, softplus);
    d = in ? d : 0.f;
    *reinterpret_cast<Two*>(at) = Two{d, d * x};
}

// A workgroup walks its segment chunk by chunk, one barrier per chunk (the LDS
// arrays alternate between two buffers).  Between two barriers the waves of its
// two halves run
//   states: the recurrence over chunk i, its sums over n into LDS
//   rows:   (d, d x), B and C of chunk i + 1 into LDS; skip and gate of chunk
//           i - 1's sums and the store of its rows; the loads of chunk i + 2
// Each SIMD holds a wave of either kind, which fill each other's latencies: 255 us
// at 8 x 4096 x 2048 (256 workgroups), the vector units issuing all the time, where
// waves that did both in turn, token group by token group, took 346 us and kept them
// busy 71 % of it.
template <typename T, int LPC, int NS, bool GATE, bool WIDE>
__global__ __launch_bounds__(128 * LPC) void scan_forward_kernel(gdr2_scan_args a, Pieces seg, uint32_t ncb, uint32_t cb_per,
                                                                 const float* starts)
{
    constexpr int NP = LPC * NS, NT = 64 * LPC, V = kScanChunk * kScanCols / NT, YLD = kScanCols + 16;
    __shared__ __align__(16) float s_b[2][kScanChunk][NP], s_c[2][kScanChunk][NP];
    __shared__ __align__(16) float s_du[2][kScanChunk / 2][kStepLd];
    __shared__ __align__(16) float s_y[2][kScanChunk][YLD];
    const uint32_t slot = blockIdx.x / ncb;
    const Piece q = uniform(piece_of(seg, slot));
    if (q.seq < 0)
        return;
    const ScanBlock blk = scan_block(a, blockIdx.x - slot * ncb, cb_per);
    const int N = (int)a.N;
    const int64_t t0 = q.index << seg.lg;
    const int64_t t1 = min(q.len, t0 + ((int64_t)1 << seg.lg));
    int buf = 0;
    if (__builtin_amdgcn_readfirstlane(threadIdx.x) < NT) {
        // ---- states
        const ScanLane l = scan_lane<LPC>(blk);
        const int s = l.s, lc = threadIdx.x / LPC, lp = step_place(lc);
        const int64_t c = l.c;
        float A2[NS], h[NS];
        load_states<NS>(a.A + c * N, s, N, l.on, A2);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            A2[i] = exponent_scale(A2[i]);
        if (starts)
            load_states<NS>(starts + ((int64_t)slot * a.C + c) * N, s, N, l.on, h);
        else
            load_states<NS>(a.h0 + (q.seq * a.C + c) * N, s, N, l.on && a.h0, h);
        const Pieces ckp{a.offsets, a.B, a.T, kScanLg};
        const int64_t ck0 = uniform(sequence_of(ckp, q.seq).first);
        for (int64_t t = t0; t < t1; t += kScanChunk, buf ^= 1) {
            if (a.h_chunks)
                store_states<NS>(a.h_chunks + ((ck0 + (t >> kScanLg)) * a.C + c) * N, s, N, l.on, h);
            lds_barrier();
            // what a token needs is read one token group ahead of its use
            float B[LPC][NS], C[LPC][NS], d[LPC], u[LPC];
#pragma unroll
            for (int k = 0; k < LPC; ++k) {
                read_states<NS>(&s_b[buf][k][s * NS], B[k]);
                read_states<NS>(&s_c[buf][k][s * NS], C[k]);
            }
#pragma unroll
            for (int k = 0; k < LPC; k += 2) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(&s_du[buf][k / 2][4 * lp]);
                d[k] = x[0], u[k] = x[1], d[k + 1] = x[2], u[k + 1] = x[3];
            }
#pragma unroll
            for (int g = 0; g < kScanChunk / LPC; ++g) {
                float p[LPC];
#pragma unroll
                for (int k = 0; k < LPC; ++k) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        h[i] = fmaf(fast_exp2(d[k] * A2[i]), h[i], u[k] * B[k][i]);
                        p[k] = i == 0 ? C[k][0] * h[0] : fmaf(C[k][i], h[i], p[k]);
                    }
                    const int next = (g + 1) * LPC + k;
                    if (next < kScanChunk) {
                        read_states<NS>(&s_b[buf][next][s * NS], B[k]);
                        read_states<NS>(&s_c[buf][next][s * NS], C[k]);
                        if (k % 2) {
                            const f32x4 x = *reinterpret_cast<const f32x4*>(&s_du[buf][next / 2][4 * lp]);
                            d[k - 1] = x[0], u[k - 1] = x[1], d[k] = x[2], u[k] = x[3];
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                s_y[buf][g * LPC + s][lc] = sum_transposed(p, s);
            }
        }
        if (t0 < t1)
            lds_barrier();
        if (a.h_out && t1 == q.len)
            store_states<NS>(a.h_out + (q.seq * a.C + c) * N, s, N, l.on, h);
    } else if (t0 < t1) {
        // ---- rows
        float bias[V], skip[V];
        channel_params<V>(a.dt_bias, blk, bias);
        channel_params<V>(a.skip, blk, skip);
        const bool soft = a.flags & GDR2_SCAN_SOFTPLUS;
        const int token = threadIdx.x / (kScanCols / V) % kScanChunk, ch = threadIdx.x % (kScanCols / V) * V;
        const int du_at = 2 * (token & 1);
        auto left_at = [&](int64_t t) { return (int)max((int64_t)0, min(t1 - t, (int64_t)kScanChunk)); };

        // rows of a chunk: dt, x (and z), B, C
        RowVec<T, V, WIDE> rt(a.dt_stride, blk), rx(a.x_stride, blk), rz(a.z_stride, blk);
        const RowVec<T, V, WIDE> ry(a.C, blk);
        Staged<T, NP, NT> rb(a.b_stride, blk.j, N), rc(a.c_stride, blk.j, N);
        const int64_t row = q.row0 + t0;
        RowWalk wt = RowWalk::at<T>(a.dt, row, a.dt_stride), wx = RowWalk::at<T>(a.x, row, a.x_stride);
        RowWalk wb = RowWalk::at<T>(a.Bt, row, a.b_stride), wc = RowWalk::at<T>(a.Ct, row, a.c_stride);
        RowWalk wz = RowWalk::at<T>(a.z, row, a.z_stride), wy = RowWalk::at<T>(a.y, row, a.C);
        auto fetch = [&](int left) {       // of no rows: reads nothing, whatever the base
            rt.load(wt, left);
            rx.load(wx, left);
            rb.load(wb, left);
            rc.load(wc, left);
            wt.advance(kScanChunk);
            wx.advance(kScanChunk);
            wb.advance(kScanChunk);
            wc.advance(kScanChunk);
            if constexpr (GATE) {
                rz.load(wz, left);
                wz.advance(kScanChunk);
            }
        };
        auto steps = [&](const RowVec<T, V, WIDE>& dt, const RowVec<T, V, WIDE>& x, bool in, int to) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                step_to_lds(dt.get(v), x.get(v), bias[v], soft, in, &s_du[to][token / 2][du_at + 4 * step_place(ch + v)]);
        };
        auto outputs = [&](const RowVec<T, V, WIDE>& x, const RowVec<T, V, WIDE>& z, int from, float (&y)[V]) {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const f32x4 p = *reinterpret_cast<const f32x4*>(&s_y[from][token][ch + v]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[v + i] = fmaf(skip[v + i], x.get(v + i), p[i]);
                    if constexpr (GATE)
                        y[v + i] *= silu_f(z.get(v + i));
                }
            }
        };
        fetch(left_at(t0));
        steps(rt, rx, token < left_at(t0), 0);
        // x, z of the previous chunk (nothing yet) and of the current one
        RowVec<T, V, WIDE> px = rx, pz = rz, cx = rx, cz = rz;
        rb.store(s_b[0]);
        rc.store(s_c[0]);
        fetch(left_at(t0 + kScanChunk));
        int64_t t = t0;
        float y[V];
        for (; t < t1; t += kScanChunk, buf ^= 1) {
            // the next chunk's rows have arrived; those after it are requested
            RowVec<T, V, WIDE> nt = rt, nx = rx, nz = rz;
            lds_barrier();
            rb.store(s_b[buf ^ 1]);
            rc.store(s_c[buf ^ 1]);
            fetch(left_at(t + 2 * kScanChunk));
            steps(nt, nx, token < left_at(t + kScanChunk), buf ^ 1);
            // (unconditional, into nothing for the first chunk: behind a branch the
            // wait for the next chunk's loads would also wait for the store)
            outputs(px, pz, buf ^ 1, y);
            ry.store(wy, t > t0 ? kScanChunk : 0, y);
            wy.advance(t > t0 ? kScanChunk : 0);
            px = cx;
            pz = cz;
            cx = nx;
            cz = nz;
        }
        lds_barrier();
        outputs(px, pz, buf ^ 1, y);
        ry.store(wy, left_at(t - kScanChunk), y);
    }
}

// (sum d, E) of every segment but the last of its sequence: whole segments.
template <typename T, int LPC, int NS, bool WIDE>
__global__ __launch_bounds__(64 * LPC) void scan_span_kernel(gdr2_scan_args a, Pieces seg, uint32_t ncb, uint32_t cb_per,
                                                             float* states, float* sums)
{
    constexpr int NP = LPC * NS, NT = 64 * LPC, V = kScanChunk * kScanCols / NT;
    __shared__ __align__(16) float s_b[2][kScanChunk][NP];
    __shared__ __align__(16) float s_du[2][kScanChunk / 2][kStepLd];
    const uint32_t slot = blockIdx.x / ncb;
    const Piece q = uniform(piece_of(seg, slot));
    const int64_t t0 = q.index << seg.lg, t1 = t0 + ((int64_t)1 << seg.lg);
    if (q.seq < 0 || t1 >= q.len)
        return;
    const ScanBlock blk = scan_block(a, blockIdx.x - slot * ncb, cb_per);
    const ScanLane l = scan_lane<LPC>(blk);
    const int s = l.s, N = (int)a.N, lc = threadIdx.x / LPC, lp = step_place(lc);
    const int64_t c = l.c;
    float A2[NS], h[NS] = {}, sum = 0.f;
    load_states<NS>(a.A + c * N, s, N, l.on, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] = exponent_scale(A2[i]);
    float bias[V];
    channel_params<V>(a.dt_bias, blk, bias);
    const bool soft = a.flags & GDR2_SCAN_SOFTPLUS;
    const int token = threadIdx.x / (kScanCols / V), ch = threadIdx.x % (kScanCols / V) * V;
    const int du_at = 2 * (token & 1);
    RowVec<T, V, WIDE> rt(a.dt_stride, blk), rx(a.x_stride, blk);
    Staged<T, NP, NT> rb(a.b_stride, blk.j, N);
    const int64_t row = q.row0 + t0;
    RowWalk wt = RowWalk::at<T>(a.dt, row, a.dt_stride), wx = RowWalk::at<T>(a.x, row, a.x_stride);
    RowWalk wb = RowWalk::at<T>(a.Bt, row, a.b_stride);
    auto fetch = [&](int left) {
        rt.load(wt, left);
        rx.load(wx, left);
        rb.load(wb, left);
        wt.advance(kScanChunk);
        wx.advance(kScanChunk);
        wb.advance(kScanChunk);
    };
    fetch(kScanChunk);
#pragma unroll
    for (int v = 0; v < V; ++v)
        step_to_lds(rt.get(v), rx.get(v), bias[v], soft, true, &s_du[0][token / 2][du_at + 4 * step_place(ch + v)]);
    rb.store(s_b[0]);
    fetch(t0 + kScanChunk < t1 ? kScanChunk : 0);
    int buf = 0;
    for (int64_t t = t0; t < t1; t += kScanChunk, buf ^= 1) {
        RowVec<T, V, WIDE> nt = rt, nx = rx;
        lds_barrier();
        rb.store(s_b[buf ^ 1]);
        fetch(t + 2 * kScanChunk < t1 ? kScanChunk : 0);
        float B[LPC][NS], d[LPC], u[LPC];
#pragma unroll
        for (int k = 0; k < LPC; ++k)
            read_states<NS>(&s_b[buf][k][s * NS], B[k]);
#pragma unroll
        for (int k = 0; k < LPC; k += 2) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&s_du[buf][k / 2][4 * lp]);
            d[k] = x[0], u[k] = x[1], d[k + 1] = x[2], u[k + 1] = x[3];
        }
#pragma unroll
        for (int g = 0; g < V; ++g) {
#pragma unroll
            for (int k = 0; k < LPC; ++k) {
                sum += d[k];
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    h[i] = fmaf(fast_exp2(d[k] * A2[i]), h[i], u[k] * B[k][i]);
                const int next = (g + 1) * LPC + k;
                if (next < kScanChunk) {
                    read_states<NS>(&s_b[buf][next][s * NS], B[k]);
                    if (k % 2) {
                        const f32x4 x = *reinterpret_cast<const f32x4*>(&s_du[buf][next / 2][4 * lp]);
                        d[k - 1] = x[0], u[k - 1] = x[1], d[k] = x[2], u[k] = x[3];
                    }
                }
                if (k == 1)
                    step_to_lds(nt.get(g), nx.get(g), bias[g], soft, true, &s_du[buf ^ 1][token / 2][du_at + 4 * step_place(ch + g)]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    store_states<NS>(states + ((int64_t)slot * a.C + c) * N, s, N, l.on, h);
    if (l.on && s == 0)
        sums[(int64_t)slot * a.C + c] = sum;
}

// Start states of a sequence's segments, written over the E of each.  One
// thread per (sequence, channel, state), whose loads run kFoldAhead segments
// ahead of the chain (32 segments of 2048 channels of 16 states: 6.9 us,
// loaded one by one 13.1).
__global__ __launch_bounds__(256) void scan_fold_kernel(gdr2_scan_args a, Pieces seg, float* states, const float* sums)
{
    const int64_t per = a.C * a.N;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.B * per)
        return;
    const int64_t seq = id / per, cn = id - seq * per, c = cn / a.N;
    const Piece q = sequence_of(seg, seq);
    const float A2 = exponent_scale(a.A[cn]);
    float h = a.h0 ? a.h0[id] : 0.f;
    const int64_t nseg = max((int64_t)1, (q.len + ((int64_t)1 << seg.lg) - 1) >> seg.lg);
    float* at = states + q.first * per + cn;
    const float* sum = sums + q.first * a.C + c;
    // the last segment has no end state to chain
    for (int64_t i = 0; i + 1 < nseg; i += kFoldAhead) {
        float e[kFoldAhead], d[kFoldAhead];
#pragma unroll
        for (int k = 0; k < kFoldAhead; ++k) {
            const bool in = i + k + 1 < nseg;
            e[k] = in ? at[(i + k) * per] : 0.f;
            d[k] = in ? sum[(i + k) * a.C] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kFoldAhead; ++k)
            if (i + k + 1 < nseg) {
                at[(i + k) * per] = h;
                h = segment_decay(A2 * d[k], h, e[k]);
            }
    }
    at[(nseg - 1) * per] = h;
}

// One token.  LPC lanes per channel, four states each; a thread keeps its
// channel's A and parameters over R sequences, whose states are all requested
// before the first is used.  The states' traffic bounds it: 256 sequences of 2048
// channels, 16 states, gated, in bf16 are 71 MB in 17.0 us, 4.2 TB/s; one sequence
// takes 4 us, a launch.
template <typename T, int LPC, int R, bool VEC>
__global__ __launch_bounds__(256) void scan_step_kernel(gdr2_scan_step_args p, uint32_t lanes)
{
    const gdr2_scan_args& a = p.s;
    const uint32_t item = blockIdx.x * 256u + threadIdx.x;
    const uint32_t rb = item / lanes, cs = item - rb * lanes;         // lanes = C * LPC rounded up to 256
    const int64_t c = cs / LPC, C = a.C, b0 = (int64_t)rb * R;
    if (b0 >= a.B)
        return;                                                       // a whole workgroup
    const int s = threadIdx.x % LPC, N = (int)a.N;
    const bool on = c < C;
    const uint32_t j = on ? (uint32_t)c / (uint32_t)(C / a.G) : 0;
    const int64_t cc = on ? c : 0;
    const T* Bt = (const T*)a.Bt + b0 * a.b_stride + j * N;
    const T* Ct = (const T*)a.Ct + b0 * a.c_stride + j * N;
    float h[R][4], A[4], Bv[R][4], Cv[R][4], x[R], dt[R], z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = on && b0 + r < a.B;
        load_states<4>(p.state + ((b0 + r) * C + cc) * N, s, N, in, h[r]);
        x[r] = in ? to_f32(((const T*)a.x)[(b0 + r) * a.x_stride + c]) : 0.f;
        dt[r] = in ? to_f32(((const T*)a.dt)[(b0 + r) * a.dt_stride + c]) : 0.f;
        z[r] = in && a.z ? to_f32(((const T*)a.z)[(b0 + r) * a.z_stride + c]) : 0.f;
        if constexpr (VEC) {
            const bool q = in && s * 4 < N;
            const f32x4 bv = q ? load4(Bt + r * a.b_stride + s * 4) : f32x4{}, cv = q ? load4(Ct + r * a.c_stride + s * 4) : f32x4{};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Bv[r][i] = bv[i];
                Cv[r][i] = cv[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool q = in && s * 4 + i < N;
                Bv[r][i] = q ? to_f32(Bt[r * a.b_stride + s * 4 + i]) : 0.f;
                Cv[r][i] = q ? to_f32(Ct[r * a.c_stride + s * 4 + i]) : 0.f;
            }
        }
    }
    load_states<4>(a.A + cc * N, s, N, on, A);
    const float bias = a.dt_bias ? a.dt_bias[cc] : 0.f, skip = a.skip ? a.skip[cc] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        A[i] = exponent_scale(A[i]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = on && b0 + r < a.B;
        const float d = step_of(dt[r] + bias, a.flags & GDR2_SCAN_SOFTPLUS), u = d * x[r];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[r][i] = fmaf(fast_exp2(d * A[i]), h[r][i], u * Bv[r][i]);
            y = fmaf(Cv[r][i], h[r][i], y);
        }
        store_states<4>(p.state + ((b0 + r) * C + cc) * N, s, N, in, h[r]);
        if constexpr (LPC >= 2)
            y += dpp_quad_xor<1>(y);
        if constexpr (LPC >= 4)
            y += dpp_quad_xor<2>(y);
        if constexpr (LPC == 8)
            y += dpp_move<0x141>(y);
        if (in && s == 0) {
            y = fmaf(skip, x[r], y);
            if (a.z)
                y *= silu_f(z[r]);
            ((T*)a.y)[(b0 + r) * C + c] = from_f32<T>(y);
        }
    }
}

struct ForwardWork {
    size_t states, sums, total;   // byte offsets, size
};

ForwardWork forward_work(const gdr2_scan_args& a, const ScanPlan& p)
{
    if (!p.split)
        return {0, 0, 0};
    const size_t st = (size_t)p.seg.slots() * a.C * a.N * 4, al = (st + 255) / 256 * 256;
    return {0, al, al + (size_t)p.seg.slots() * a.C * 4};
}

template <typename T, int LPC, int NS, bool WIDE>
hipError_t forward_t(const gdr2_scan_args& a, hipStream_t stream)
{
    const ScanPlan p = scan_plan(a, false);
    const ForwardWork w = forward_work(a, p);
    const dim3 grid((unsigned)(p.seg.slots() * p.ncb)), block(64 * LPC);
    const uint32_t ncb = (uint32_t)p.ncb, cb_per = (uint32_t)p.cb_per;
    float* states = nullptr;
    if (p.split) {
        states = (float*)((char*)a.workspace + w.states);
        float* sums = (float*)((char*)a.workspace + w.sums);
        hipLaunchKernelGGL((scan_span_kernel<T, LPC, NS, WIDE>), grid, block, 0, stream, a, p.seg, ncb, cb_per, states, sums);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL(scan_fold_kernel, dim3((unsigned)ceil_div(a.B * a.C * a.N, 256)), dim3(256), 0, stream, a, p.seg,
                           states, sums);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    if (a.z)
        hipLaunchKernelGGL((scan_forward_kernel<T, LPC, NS, true, WIDE>), grid, dim3(128 * LPC), 0, stream, a, p.seg, ncb, cb_per, states);
    else
        hipLaunchKernelGGL((scan_forward_kernel<T, LPC, NS, false, WIDE>), grid, dim3(128 * LPC), 0, stream, a, p.seg, ncb, cb_per, states);
    return hipGetLastError();
}

template <typename T, int LPC, int NS>
hipError_t forward_w(const gdr2_scan_args& a, hipStream_t stream)
{
    return scan_wide(a, kScanChunk / LPC) ? forward_t<T, LPC, NS, true>(a, stream) : forward_t<T, LPC, NS, false>(a, stream);
}

// Lanes per channel of the step; a sequence's lanes, in whole workgroups.
int step_lpc(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : 8; }
int64_t step_lanes(int64_t C, int lpc) { return ceil_div(C * lpc, 256) * 256; }

// Sequences per thread: two once that leaves four waves per SIMD (256 x 2048
// channels, 16 states: 16.8 us when all were timed; one 19.4, four 20.0, eight 26;
// streaming accesses to the state 22), else one.
int step_sequences(const gdr2_scan_args& a)
{
    return a.B / 2 * a.C * step_lpc(a.N) >= (int64_t)device_cu_count() * 4 * 4 * 64 ? 2 : 1;
}

template <typename T, int LPC, int R, bool VEC>
hipError_t step_r(const gdr2_scan_step_args& a, hipStream_t stream)
{
    const int64_t lanes = step_lanes(a.s.C, LPC);
    hipLaunchKernelGGL((scan_step_kernel<T, LPC, R, VEC>), dim3((unsigned)(ceil_div(a.s.B, R) * (lanes / 256))), dim3(256), 0,
                       stream, a, (uint32_t)lanes);
    return hipGetLastError();
}
template <typename T, int LPC>
hipError_t step_t(const gdr2_scan_step_args& a, hipStream_t stream)
{
    const int64_t e = sizeof(T);
    auto ok = [&](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % (4 * e) == 0 && ld % 4 == 0; };
    const bool vec = a.s.N % 4 == 0 && ok(a.s.Bt, a.s.b_stride) && ok(a.s.Ct, a.s.c_stride);
    if (step_sequences(a.s) == 2)
        return vec ? step_r<T, LPC, 2, true>(a, stream) : step_r<T, LPC, 2, false>(a, stream);
    return vec ? step_r<T, LPC, 1, true>(a, stream) : step_r<T, LPC, 1, false>(a, stream);
}

template <typename T>
hipError_t step_n(const gdr2_scan_step_args& a, hipStream_t stream)
{
    switch (step_lpc(a.s.N)) {
    case 1: return step_t<T, 1>(a, stream);
    case 2: return step_t<T, 2>(a, stream);
    case 4: return step_t<T, 4>(a, stream);
    default: return step_t<T, 8>(a, stream);
    }
}

}  // namespace

// How a call is cut into segments.
// One segment per sequence where that keeps the compute units busy, for the span
// pass repeats most of the work: forwards from 9/16 of a workgroup per unit on (2048
// channels, 16 states, 4096 tokens: 128 workgroups 251 us whole, 226 in segments;
// 160: 251 and 274; 256: 258 and 417), backwards, where two workgroups share a
// unit, from 7/4 (2048 tokens: 256 workgroups 848 us whole, 684 in segments; 448:
// 1108 and 1149; 512: 1128 and 1327).  Otherwise the longest segments that give
// every unit four workgroups, two rounds of what is resident, at least 128 tokens:
// 1 x 32768 tokens (32 channel blocks) 426 us with 1024 workgroups, 438 us with 512.
// A packed batch is cut at twice its mean length in any case: the host does
// not know the lengths, one sequence may hold nearly all rows, and sequences
// that fit one segment skip the span pass.  Some of its slots are idle and some
// segments short, so whole segments have to give a workgroup per unit there (9
// sequences, 5003 rows of 1002 channels, four draws of the lengths: 76 to 80 us,
// with the dense rule 77 to 318).
ScanPlan scan_plan(const gdr2_scan_args& a, bool backward)
{
    ScanPlan p;
    p.cb_per = ceil_div(a.C / a.G, kScanCols);
    p.ncb = p.cb_per * a.G;
    int whole = kScanLg;                      // a segment that holds any sequence
    while (((int64_t)1 << whole) < a.T)
        ++whole;
    const int shortest = std::min(whole, kScanLg + 2);
    int lg = whole;
    auto groups = [&](int g) { return Pieces{a.offsets, a.B, a.T, g}.slots() * p.ncb; };
    if (a.algo == GDR2_ALGO_SEGMENTED) {
        lg = std::min(whole, kScanLg + 1);
    } else if (a.algo == GDR2_ALGO_AUTO) {
        if (a.offsets)
            while (lg > shortest && ((int64_t)1 << (lg - 1)) >= 2 * ceil_div(a.T, std::max(a.B, (int64_t)1)))
                --lg;
        const int64_t cus = device_cu_count();
        if (16 * groups(lg) < (backward ? 28 : a.offsets ? 16 : 9) * cus)
            while (lg > shortest && groups(lg) < 4 * cus)
                --lg;
    }
    p.seg = Pieces{a.offsets, a.B, a.T, lg};
    p.split = lg < whole;
    return p;
}

int64_t scan_launch_groups(const gdr2_scan_args& a, ScanCall call)
{
    if (call == ScanCall::Step) {
        const int64_t lanes = step_lanes(a.C, step_lpc(a.N));
        return ceil_div(a.B, step_sequences(a)) * (lanes / 256);
    }
    const bool backward = call == ScanCall::Backward;
    const ScanPlan p = scan_plan(a, backward);
    int64_t n;
    if (__builtin_mul_overflow(p.seg.slots(), p.ncb, &n) || n >= kMaxGroups)
        return kMaxGroups;
    // 64 threads for every lane of a channel, twice that forwards
    n *= (a.N > 16 ? 2 : 1) * (backward ? 1 : 2);
    if (p.split)
        n = std::max(n, ceil_div(a.B * a.C * a.N, 256));
    if (backward) {
        const double sums = (double)(a.offsets ? a.T : a.B * a.T) * (double)(a.G * 2 * a.N) / 256.0;
        n = std::max(n, sums >= (double)kMaxGroups ? kMaxGroups : (int64_t)sums + 1);
    }
    return n;
}

size_t scan_workspace_bytes(const gdr2_scan_args& a) { return forward_work(a, scan_plan(a, false)).total; }

// Lanes per channel and states per lane.  16 states run on 4 lanes of 4, which need
// half the LDS reads of 8 lanes of 2; 32 states need the 8 lanes for their registers.
hipError_t launch_scan_forward(const gdr2_scan_args& a, hipStream_t stream)
{
    const bool bf = a.dtype == GDR2_BF16;
    if (a.N <= 8)
        return bf ? forward_w<bf16, 4, 2>(a, stream) : forward_w<float, 4, 2>(a, stream);
    if (a.N <= 16)
        return bf ? forward_w<bf16, 4, 4>(a, stream) : forward_w<float, 4, 4>(a, stream);
    return bf ? forward_w<bf16, 8, 4>(a, stream) : forward_w<float, 8, 4>(a, stream);
}

hipError_t launch_scan_step(const gdr2_scan_step_args& a, hipStream_t stream)
{
    return a.s.dtype == GDR2_BF16 ? step_n<bf16>(a, stream) : step_n<float>(a, stream);
}

}  // namespace gdr2
