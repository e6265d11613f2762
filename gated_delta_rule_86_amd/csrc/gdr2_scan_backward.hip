// gdr2_scan_backward.hip -- gradients of the selective state space scan.
//
// With dv = dy silu(z) and lam_t the gradient of h_t:
//   lam_t = dv_t C_t + a_{t+1} lam_{t+1},   a_t = exp(d_t A)
//   du = sum_n lam B,  dx = d du + skip dv,  dB = sum_c lam d x,  dC = sum_c dv h
//   q = lam a h_{t-1},  dd = x du + sum_n q A,  ddt = dd sigmoid(raw),  dA = sum d q
//   dz = dy v silu'(z),  dskip = sum dv x,  dh0 = a_0 lam_0
// The states come from the forward's record of every 32nd one: a chunk's
// states are formed again from its start, kSub tokens at a time, and stay in
// registers with their decays while those tokens are walked backwards.
//
// The arithmetic bounds it: about 104 vector operations per token and wave of 16
// channels (26.8 thousand for 256 tokens).  4 x 2048 x 2048 channels of 16 states,
// gated: 278 us for the main pass, 53 us for the segments' gradients.  The sums
// over channels (dB, dC) are the expensive ones: a transposing reduction
// over the channels of a wave, LDS over the waves, one partial row per channel
// block, added by a last kernel in block order.  The sums over tokens (dA,
// dskip, ddt_bias) stay in registers for a whole segment and leave as one
// partial row per segment.
#include "gdr2_scan.h"

namespace gdr2 {

namespace {

constexpr int kSub = 8;                       // tokens whose states are held
constexpr int kSubs = kScanChunk / kSub;

// Sum of v[k][i], four tokens k, over the channels of a wave: lanes of row
// r = lane / 16 return token k = r.  (Rounds over lane bits 5 and 4 halve the
// values held; bit 3, and bit 2 with four lanes a channel, are rotations
// within the row.)
template <int LPC, int NS>
__device__ __forceinline__ void channel_sum(const float (&v)[4][NS], float (&r)[NS])
{
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        float x = pair_sum16(pair_sum32(v[0][i], v[2][i]), pair_sum32(v[1][i], v[3][i]));
        x += dpp_move<0x128>(x);          // row_ror:8
        if constexpr (LPC == 4)
            x += dpp_move<0x124>(x);      // row_ror:4
        r[i] = x;
    }
}

// sum_transposed with its values arriving from k = LPC - 1 down to 0: of eight
// values the upper four are combined with the lower ones as these come.
template <int LPC> struct TransposedSum {
    float q[4], up[4];
    __device__ __forceinline__ void put(int k, float p, int s)   // k is known after unrolling
    {
        if (LPC == 4)
            q[k] = p;
        else if (k >= 4)
            up[k - 4] = p;
        else
            q[k] = (s & 4 ? up[k] : p) + dpp_move<0x141>(s & 4 ? p : up[k]);
    }
    __device__ __forceinline__ float get(int s) const { return sum_transposed(q, s); }
};

// Floats of one segment's row of token sums (rows start on 16 bytes).
__host__ __device__ inline int64_t sums_ld(int64_t C, int64_t N) { return (C * (N + 2) + 3) / 4 * 4; }

struct BackwardPtrs {
    float* parts;       // [ncb][rows][2][N]: dB, dC of one channel block
    float* sums;        // [slots][sums_ld]: dA [C][N], dskip [C], ddt_bias [C]
    const float* lam;   // [slots][C][N] gradients entering each segment from behind, or NULL
};

// One chunk at a time, last to first:
//   rows:   d, d x, dv of the chunk into LDS       | barrier
//   states: forwards for the states, backwards for the gradients, the sums over
//           n into the places of d x, dv, and the sums over channels | barrier
//   rows:   dx, ddt, dz from the sums; dB, dC over the waves
template <typename T, int LPC, int NS, bool GATE, bool WIDE>
__global__ __launch_bounds__(64 * LPC, 2) void scan_backward_kernel(gdr2_scan_bwd_args p, Pieces seg, uint32_t ncb, uint32_t cb_per,
                                                                 BackwardPtrs w)
{
    constexpr int NP = LPC * NS, NT = 64 * LPC, V = kScanChunk * kScanCols / NT, NW = NT / 64;
    const gdr2_scan_args& a = p.f;
    __shared__ __align__(16) float s_b[kScanChunk][NP], s_c[kScanChunk][NP];
    __shared__ __align__(16) f32x4 s_tok[kScanChunk][kScanCols];          // d, d x, dv, - and then d, du, qA, v
    __shared__ __align__(16) float s_red[2][NW][kScanChunk][NP];
    __shared__ __align__(16) float s_h[kSubs - 1][NT][NS];               // before sub-chunks 1, 2, ..
    const uint32_t slot = blockIdx.x / ncb, cb = blockIdx.x - slot * ncb;
    const Piece q = uniform(piece_of(seg, slot));
    const ScanBlock blk = scan_block(a, cb, cb_per);
    const ScanLane l = scan_lane<LPC>(blk);
    const int s = l.s, N = (int)a.N, lp = step_place(threadIdx.x / LPC), wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t C = a.C, c = l.c;
    const int token = threadIdx.x / (kScanCols / V), ch = threadIdx.x % (kScanCols / V) * V;
    float* sums = w.sums + (int64_t)slot * sums_ld(C, N);
    float dA[NS] = {}, dskip[V] = {}, dbias[V] = {};
    const int64_t t0 = q.seq < 0 ? 0 : q.index << seg.lg;
    const int64_t t1 = q.seq < 0 ? 0 : min(q.len, t0 + ((int64_t)1 << seg.lg));
    float lam[NS] = {};
    if (q.seq >= 0) {
        if (w.lam)
            load_states<NS>(w.lam + ((int64_t)slot * C + c) * N, s, N, l.on, lam);
        else
            load_states<NS>(p.dh_out + (q.seq * C + c) * N, s, N, l.on && p.dh_out, lam);
    }
    if (t0 < t1) {
        float A[NS], A2[NS];
        load_states<NS>(a.A + c * N, s, N, l.on, A);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            A2[i] = exponent_scale(A[i]), A[i] = finite(A[i]);
        float bias[V], skips[V];
        channel_params<V>(a.dt_bias, blk, bias);
        channel_params<V>(a.skip, blk, skips);
        const bool soft = a.flags & GDR2_SCAN_SOFTPLUS;
        const Pieces ckp{a.offsets, a.B, a.T, kScanLg};
        const int64_t ck0 = uniform(sequence_of(ckp, q.seq).first);
        const int64_t rows = a.offsets ? a.T : a.B * a.T;
        float* part = w.parts + (int64_t)cb * rows * 2 * N;

        int64_t t = t0 + ((t1 - t0 - 1) >> kScanLg << kScanLg);
        const int64_t row = q.row0 + t;
        RowVec<T, V, WIDE> rt(a.dt_stride, blk), rx(a.x_stride, blk), rd(C, blk), rz(a.z_stride, blk);
        const RowVec<T, V, WIDE> ro(C, blk);
        Staged<T, NP, NT> rb(a.b_stride, blk.j, N), rc(a.c_stride, blk.j, N);
        RowWalk wt = RowWalk::at<T>(a.dt, row, a.dt_stride), wx = RowWalk::at<T>(a.x, row, a.x_stride);
        RowWalk wb = RowWalk::at<T>(a.Bt, row, a.b_stride), wc = RowWalk::at<T>(a.Ct, row, a.c_stride);
        RowWalk wz = RowWalk::at<T>(a.z, row, a.z_stride), wd = RowWalk::at<T>(p.dy, row, C);
        RowWalk wdx = RowWalk::at<T>(p.dx, row, C), wdt = RowWalk::at<T>(p.ddt, row, C), wdz = RowWalk::at<T>(p.dz, row, C);
        auto fetch = [&](int left) {
            rt.load(wt, left);
            rx.load(wx, left);
            rd.load(wd, left);
            rb.load(wb, left);
            rc.load(wc, left);
            wt.advance(-kScanChunk);
            wx.advance(-kScanChunk);
            wd.advance(-kScanChunk);
            wb.advance(-kScanChunk);
            wc.advance(-kScanChunk);
            if constexpr (GATE) {
                rz.load(wz, left);
                wz.advance(-kScanChunk);
            }
        };
        int left = (int)(t1 - t);
        fetch(left);
        float h0[NS];
        load_states<NS>(a.h_chunks + ((ck0 + (t >> kScanLg)) * C + c) * N, s, N, l.on, h0);
        for (;; t -= kScanChunk) {
            // rows of this chunk
            rb.store(s_b);
            rc.store(s_c);
            const RowVec<T, V, WIDE> xt = rt, xx = rx, xd = rd, xz = rz;
            const bool in = token < left;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float raw = xt.get(v) + bias[v], x = xx.get(v);
                float d = step_of(raw, soft), dv = xd.get(v);
                if constexpr (GATE)
                    dv *= silu_f(xz.get(v));
                d = in ? d : 0.f;
                dv = in ? dv : 0.f;
                s_tok[token][step_place(ch + v)] = f32x4{d, d * x, dv, 0.f};
            }
            lds_barrier();
            const bool more = t > t0;
            fetch(more ? kScanChunk : 0);
            // Tokens are read from LDS two ahead, in rings by parity; the scheduling
            // barriers keep the compiler from gathering the reads in front of their uses.
            f32x4 tk[2];
            float Bq[2][NS], Cq[2][NS];
            auto read = [&](int tt, int r) {
                tk[r] = s_tok[tt][lp];
                read_states<NS>(&s_b[tt][s * NS], Bq[r]);
            };
            // the states before every kSub tokens
            {
                float h[NS];
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    h[i] = h0[i];
                read(0, 0);
                read(1, 1);
#pragma unroll 1
                for (int b = 0; b < kSubs - 1; ++b) {
#pragma unroll
                    for (int k = 0; k < kSub; ++k) {
#pragma unroll
                        for (int i = 0; i < NS; ++i)
                            h[i] = fmaf(fast_exp2(tk[k & 1][0] * A2[i]), h[i], tk[k & 1][1] * Bq[k & 1][i]);
                        read(b * kSub + k + 2, k & 1);
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int i = 0; i < NS; ++i)
                        s_h[b][threadIdx.x][i] = h[i];
                }
            }
            // (the rings now hold the last sub-chunk's first two tokens)
#pragma unroll 1
            for (int b = kSubs - 1; b >= 0; --b) {
                const int first = b * kSub, before = b > 0 ? first - kSub : 0;
                float av[kSub][NS], hv[kSub + 1][NS];
                if (b > 0) {
                    read_states<NS>(&s_h[b - 1][threadIdx.x][0], hv[0]);
                } else {
#pragma unroll
                    for (int i = 0; i < NS; ++i)
                        hv[0][i] = h0[i];
                }
#pragma unroll
                for (int k = 0; k < kSub; ++k) {
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        av[k][i] = fast_exp2(tk[k & 1][0] * A2[i]);
                        hv[k + 1][i] = fmaf(av[k][i], hv[k][i], tk[k & 1][1] * Bq[k & 1][i]);
                    }
                    if (k + 2 < kSub)
                        read(first + k + 2, k & 1);
                    else
                        read_states<NS>(&s_c[first + k][s * NS], Cq[k & 1]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int g = kSub / LPC - 1; g >= 0; --g) {
                    TransposedSum<LPC> su, sa, sv;
                    float vb[4][NS], vc[4][NS];
#pragma unroll
                    for (int k = LPC - 1; k >= 0; --k) {
                        const int kk = g * LPC + k, r = kk & 1;
                        float pu = 0.f, pa = 0.f, pv = 0.f;
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            const float gr = fmaf(Cq[r][i], tk[r][2], lam[i]);
                            vc[k % 4][i] = tk[r][2] * hv[kk + 1][i];
                            vb[k % 4][i] = gr * tk[r][1];
                            lam[i] = gr * av[kk][i];
                            const float qq = lam[i] * hv[kk][i];
                            dA[i] = fmaf(qq, tk[r][0], dA[i]);
                            pu = i == 0 ? gr * Bq[r][0] : fmaf(gr, Bq[r][i], pu);
                            pa = i == 0 ? qq * A[0] : fmaf(qq, A[i], pa);
                            if constexpr (GATE)
                                pv = i == 0 ? Cq[r][0] * hv[kk + 1][0] : fmaf(Cq[r][i], hv[kk + 1][i], pv);
                        }
                        if (kk >= 2) {
                            read(first + kk - 2, r);
                            read_states<NS>(&s_c[first + kk - 2][s * NS], Cq[r]);
                        } else {
                            read(before + kk, r);
                        }
                        su.put(k, pu, s);
                        sa.put(k, pa, s);
                        if constexpr (GATE)
                            sv.put(k, pv, s);
                        if (k % 4 == 0) {
                            float xb[NS], xc[NS];
                            channel_sum<LPC, NS>(vb, xb);
                            channel_sum<LPC, NS>(vc, xc);
                            // (the lanes of a row that share s hold and write the same value)
                            const int at = first + kk + (lane >> 4);
#pragma unroll
                            for (int i = 0; i < NS; ++i) {
                                s_red[0][wave][at][s * NS + i] = xb[i];
                                s_red[1][wave][at][s * NS + i] = xc[i];
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    // lane s: token s of the group, whose values every lane has read
                    float* at = (float*)&s_tok[first + g * LPC + s][lp];
                    at[1] = su.get(s);
                    at[2] = sa.get(s);
                    if constexpr (GATE)
                        at[3] = sv.get(s);
                }
            }
            if (more)
                load_states<NS>(a.h_chunks + ((ck0 + (t >> kScanLg) - 1) * C + c) * N, s, N, l.on, h0);
            lds_barrier();
            float dx[V], ddt[V], dz[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const f32x4 tk = s_tok[token][step_place(ch + v)];
                const float x = xx.get(v), dy = xd.get(v), raw = xt.get(v) + bias[v], skip = skips[v];
                float dv = dy;
                if constexpr (GATE) {
                    const float z = xz.get(v), sg = sigmoid_f(z);
                    dv = dy * z * sg;
                    dz[v] = dy * fmaf(skip, x, tk[3]) * (sg * fmaf(z, 1.f - sg, 1.f));
                }
                float dd = fmaf(x, tk[1], tk[2]);
                dd = soft ? dd * sigmoid_f(raw) : dd;
                dx[v] = fmaf(tk[0], tk[1], skip * dv);
                ddt[v] = dd;
                // (rows past the sequence read as zero: dv = x = 0)
                dskip[v] = fmaf(dv, x, dskip[v]);
                dbias[v] += in ? dd : 0.f;
            }
            ro.store(wdx, left, dx);
            ro.store(wdt, left, ddt);
            if constexpr (GATE)
                ro.store(wdz, left, dz);
            wdx.advance(-kScanChunk);
            wdt.advance(-kScanChunk);
            wdz.advance(-kScanChunk);
            for (int e = threadIdx.x; e < 2 * kScanChunk * NP; e += NT) {
                const int r = e / (2 * NP), which = e / NP % 2, n = e % NP;
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < NW; ++k)
                    x += s_red[which][k][r][n];
                if (r < left && n < N)
                    part[((q.row0 + t + r) * 2 + which) * N + n] = x;
            }
            if (!more)
                break;
            left = kScanChunk;
            lds_barrier();
        }
    }
    if (q.seq >= 0 && p.dh0 && q.index == 0)
        store_states<NS>(p.dh0 + (q.seq * C + c) * N, s, N, l.on, lam);
    store_states<NS>(sums + c * N, s, N, l.on, dA);
    // dskip and ddt_bias over the threads that share their channels, in token order
    lds_barrier();
    f32x4* both = &s_tok[0][0];
#pragma unroll
    for (int v = 0; v < V; ++v)
        both[token * kScanCols + ch + v] = f32x4{dskip[v], dbias[v], 0.f, 0.f};
    lds_barrier();
    if ((int)threadIdx.x < blk.n) {
        float x = 0.f, y = 0.f;
        for (int k = 0; k < kScanChunk; ++k) {
            const f32x4 e = both[k * kScanCols + threadIdx.x];
            x += e[0];
            y += e[1];
        }
        sums[C * N + blk.c0 + threadIdx.x] = x;
        sums[C * (N + 1) + blk.c0 + threadIdx.x] = y;
    }
}

// Per segment but the first of its sequence: the gradient of its start state
// when none enters from behind, and sum d.
template <typename T, int LPC, int NS, bool GATE, bool WIDE>
__global__ __launch_bounds__(64 * LPC) void scan_backward_span_kernel(gdr2_scan_bwd_args p, Pieces seg, uint32_t ncb,
                                                                      uint32_t cb_per, float* states, float* sums)
{
    constexpr int NP = LPC * NS, NT = 64 * LPC, V = kScanChunk * kScanCols / NT;
    const gdr2_scan_args& a = p.f;
    __shared__ __align__(16) float s_c[2][kScanChunk][NP];
    __shared__ __align__(16) float s_du[2][kScanChunk / 2][kStepLd];      // d, dv as the forward's d, d x
    const uint32_t slot = blockIdx.x / ncb;
    const Piece q = uniform(piece_of(seg, slot));
    if (q.seq < 0 || q.index == 0)
        return;
    const ScanBlock blk = scan_block(a, blockIdx.x - slot * ncb, cb_per);
    const ScanLane l = scan_lane<LPC>(blk);
    const int s = l.s, N = (int)a.N, lp = step_place(threadIdx.x / LPC);
    const int64_t C = a.C, c = l.c;
    float A2[NS], lam[NS] = {}, sum = 0.f;
    load_states<NS>(a.A + c * N, s, N, l.on, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] = exponent_scale(A2[i]);
    float bias[V];
    channel_params<V>(a.dt_bias, blk, bias);
    const bool soft = a.flags & GDR2_SCAN_SOFTPLUS;
    const int token = threadIdx.x / (kScanCols / V), ch = threadIdx.x % (kScanCols / V) * V;
    const int64_t t0 = q.index << seg.lg;
    const int64_t t1 = min(q.len, t0 + ((int64_t)1 << seg.lg));
    int64_t t = t0 + ((t1 - t0 - 1) >> kScanLg << kScanLg);
    const int64_t row = q.row0 + t;
    RowVec<T, V, WIDE> rt(a.dt_stride, blk), rd(C, blk), rz(a.z_stride, blk);
    Staged<T, NP, NT> rc(a.c_stride, blk.j, N);
    RowWalk wt = RowWalk::at<T>(a.dt, row, a.dt_stride), wd = RowWalk::at<T>(p.dy, row, C);
    RowWalk wz = RowWalk::at<T>(a.z, row, a.z_stride), wc = RowWalk::at<T>(a.Ct, row, a.c_stride);
    auto fetch = [&](int left) {
        rt.load(wt, left);
        rd.load(wd, left);
        rc.load(wc, left);
        wt.advance(-kScanChunk);
        wd.advance(-kScanChunk);
        wc.advance(-kScanChunk);
        if constexpr (GATE) {
            rz.load(wz, left);
            wz.advance(-kScanChunk);
        }
    };
    int left = (int)(t1 - t), buf = 0;
    fetch(left);
    for (; t >= t0; t -= kScanChunk, buf ^= 1) {
        rc.store(s_c[buf]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            typedef float Two __attribute__((ext_vector_type(2)));
            const float raw = rt.get(v) + bias[v];
            float d = step_of(raw, soft), dv = rd.get(v);
            if constexpr (GATE)
                dv *= silu_f(rz.get(v));
            d = token < left ? d : 0.f;
            dv = token < left ? dv : 0.f;
            *reinterpret_cast<Two*>(&s_du[buf][token / 2][4 * step_place(ch + v) + 2 * (token & 1)]) = Two{d, dv};
        }
        left = kScanChunk;
        fetch(t > t0 ? kScanChunk : 0);
        lds_barrier();
#pragma unroll
        for (int tt = kScanChunk - 2; tt >= 0; tt -= 2) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&s_du[buf][tt / 2][4 * lp]);
            sum += x[0] + x[2];
            float C0[NS], C1[NS];
            read_states<NS>(&s_c[buf][tt][s * NS], C0);
            read_states<NS>(&s_c[buf][tt + 1][s * NS], C1);
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                lam[i] = fmaf(C1[i], x[3], lam[i]) * fast_exp2(x[2] * A2[i]);
                lam[i] = fmaf(C0[i], x[1], lam[i]) * fast_exp2(x[0] * A2[i]);
            }
        }
    }
    store_states<NS>(states + ((int64_t)slot * C + c) * N, s, N, l.on, lam);
    if (l.on && s == 0)
        sums[(int64_t)slot * C + c] = sum;
}

// The gradient entering each segment from behind, written over the span
// pass's states.
__global__ __launch_bounds__(256) void scan_backward_fold_kernel(gdr2_scan_bwd_args p, Pieces seg, float* states,
                                                                 const float* sums)
{
    const gdr2_scan_args& a = p.f;
    const int64_t per = a.C * a.N;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.B * per)
        return;
    const int64_t seq = id / per, cn = id - seq * per, c = cn / a.N;
    const Piece q = sequence_of(seg, seq);
    const float A2 = exponent_scale(a.A[cn]);
    float lam = p.dh_out ? p.dh_out[id] : 0.f;
    const int64_t nseg = max((int64_t)1, (q.len + ((int64_t)1 << seg.lg) - 1) >> seg.lg);
    float* at = states + q.first * per + cn;
    const float* sum = sums + q.first * a.C + c;
    // the first segment has nothing before it to pass its gradient to
    for (int64_t i = nseg - 1; i > 0; i -= kFoldAhead) {
        float e[kFoldAhead], d[kFoldAhead];
#pragma unroll
        for (int k = 0; k < kFoldAhead; ++k) {
            const bool in = i - k > 0;
            e[k] = in ? at[(i - k) * per] : 0.f;
            d[k] = in ? sum[(i - k) * a.C] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kFoldAhead; ++k)
            if (i - k > 0) {
                at[(i - k) * per] = lam;
                lam = segment_decay(A2 * d[k], lam, e[k]);
            }
    }
    at[0] = lam;
}

// dB and dC: the channel blocks' partial sums of each row, in block order.
template <typename T>
__global__ __launch_bounds__(256) void scan_rows_sum_kernel(gdr2_scan_bwd_args p, const float* parts, int64_t rows,
                                                            uint32_t cb_per)
{
    const gdr2_scan_args& a = p.f;
    const uint32_t N = (uint32_t)a.N, G = (uint32_t)a.G, id = blockIdx.x * 256u + threadIdx.x;
    const uint32_t g = id / (2 * N), e = id - g * 2 * N, row = g / G, j = g - row * G;   // e: dB, then dC
    if (row >= rows)
        return;
    if (a.offsets) {
        // rows of no sequence: before the first or behind the last
        const Pieces pc{a.offsets, a.B, a.T, 0};
        if (row < clamp_offset(pc, 0) || row >= clamp_offset(pc, a.B))
            return;
    }
    const float* at = parts + ((int64_t)j * cb_per * rows + row) * 2 * N + e;
    float x = 0.f;
#pragma unroll 8
    for (uint32_t i = 0; i < cb_per; ++i)
        x += at[(int64_t)i * rows * 2 * N];
    T* to = (T*)(e < N ? p.dBt : p.dCt);
    to[(int64_t)g * N + (e < N ? e : e - N)] = from_f32<T>(x);
}

struct BackwardWork {
    size_t parts, sums, lam, span, total;
};

BackwardWork backward_work(const gdr2_scan_bwd_args& p, const ScanPlan& pl)
{
    const gdr2_scan_args& a = p.f;
    const int64_t rows = a.offsets ? a.T : a.B * a.T, slots = pl.seg.slots();
    auto al = [](size_t x) { return (x + 255) / 256 * 256; };
    BackwardWork w;
    w.parts = 0;
    w.sums = al((size_t)pl.ncb * rows * 2 * a.N * 4);
    w.lam = w.sums + al((size_t)slots * sums_ld(a.C, a.N) * 4);
    w.span = w.lam + (pl.split ? al((size_t)slots * a.C * a.N * 4) : 0);
    w.total = w.span + (pl.split ? (size_t)slots * a.C * 4 : 0);
    return w;
}

template <typename T, int LPC, int NS, bool GATE, bool WIDE>
hipError_t backward_t(const gdr2_scan_bwd_args& p, hipStream_t stream)
{
    const gdr2_scan_args& a = p.f;
    const ScanPlan pl = scan_plan(a, true);
    const BackwardWork w = backward_work(p, pl);
    char* ws = (char*)p.workspace;
    const dim3 grid((unsigned)(pl.seg.slots() * pl.ncb)), block(64 * LPC);
    const uint32_t ncb = (uint32_t)pl.ncb, cb_per = (uint32_t)pl.cb_per;
    const int64_t rows = a.offsets ? a.T : a.B * a.T;
    BackwardPtrs ptr{(float*)(ws + w.parts), (float*)(ws + w.sums), nullptr};
    hipError_t e;
    if (pl.split) {
        float* lam = (float*)(ws + w.lam);
        float* span = (float*)(ws + w.span);
        hipLaunchKernelGGL((scan_backward_span_kernel<T, LPC, NS, GATE, WIDE>), grid, block, 0, stream, p, pl.seg, ncb, cb_per,
                           lam, span);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        hipLaunchKernelGGL(scan_backward_fold_kernel, dim3((unsigned)ceil_div(a.B * a.C * a.N, 256)), dim3(256), 0, stream, p,
                           pl.seg, lam, span);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        ptr.lam = lam;
    }
    hipLaunchKernelGGL((scan_backward_kernel<T, LPC, NS, GATE, WIDE>), grid, block, 0, stream, p, pl.seg, ncb, cb_per, ptr);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    if (rows > 0) {
        hipLaunchKernelGGL((scan_rows_sum_kernel<T>), dim3((unsigned)ceil_div(rows * a.G * 2 * a.N, 256)), dim3(256), 0, stream,
                           p, ptr.parts, rows, cb_per);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    return launch_column_sum(ptr.sums, pl.seg.slots(), sums_ld(a.C, a.N), {p.dA, a.C * a.N}, {p.dskip, a.C}, {p.ddt_bias, a.C}, stream);
}

template <typename T, int LPC, int NS>
hipError_t backward_w(const gdr2_scan_bwd_args& p, hipStream_t stream)
{
    constexpr int V = kScanChunk / LPC;
    const int64_t e = sizeof(T);
    auto ok = [&](const void* q) { return !q || reinterpret_cast<uintptr_t>(q) % (V * e) == 0; };
    const bool wide = scan_wide(p.f, V) && ok(p.dy) && ok(p.dx) && ok(p.ddt) && ok(p.dz);
    if (p.f.z)
        return wide ? backward_t<T, LPC, NS, true, true>(p, stream) : backward_t<T, LPC, NS, true, false>(p, stream);
    return wide ? backward_t<T, LPC, NS, false, true>(p, stream) : backward_t<T, LPC, NS, false, false>(p, stream);
}

}  // namespace

size_t scan_backward_workspace_bytes(const gdr2_scan_bwd_args& p) { return backward_work(p, scan_plan(p.f, true)).total; }

hipError_t launch_scan_backward(const gdr2_scan_bwd_args& p, hipStream_t stream)
{
    const gdr2_scan_args& a = p.f;
    if (a.B == 0)      // no rows: zeros are all there is to write
        return launch_column_sum(nullptr, 0, 0, {p.dA, a.C * a.N}, {p.dskip, a.C}, {p.ddt_bias, a.C}, stream);
    const bool bf = a.dtype == GDR2_BF16;
    if (a.N <= 8)
        return bf ? backward_w<bf16, 4, 2>(p, stream) : backward_w<float, 4, 2>(p, stream);
    if (a.N <= 16)
        return bf ? backward_w<bf16, 4, 4>(p, stream) : backward_w<float, 4, 4>(p, stream);
    return bf ? backward_w<bf16, 8, 4>(p, stream) : backward_w<float, 8, 4>(p, stream);
}

}  // namespace gdr2
