// gdr2_scan_backward.hip -- gradients of the selective state space scan.
//
// With dv = dy silu(z) and lam_t the gradient of h_t:
//   lam_t = dv_t C_t + a_{t+1} lam_{t+1},   a_t = exp(d_t A)
//   du = sum_n lam B,  dx = d du + skip dv,  dB = sum_c lam d x,  dC = sum_c dv h
//   q = lam a h_{t-1},  dd = x du + sum_n q A,  ddt = dd sigmoid(raw),  dA = sum d q
//   dz = dy v silu'(z),  dskip = sum dv x,  dh0 = a_0 lam_0
// The states come from the forward's record of every 32nd one: a chunk's
// states are formed again from its start, SUB tokens at a time, and stay in
// registers with their decays while the chunk is walked backwards.
//
// The sums over channels (dB, dC) are the expensive ones: per token group a
// transposing reduction over the 16 channels of a wave, then LDS over the
// waves, then one partial row per channel block, added by a last kernel in
// block order.  The sums over tokens (dA, dskip, ddt_bias) stay in registers
// for a whole segment and leave as one partial row per segment.
#include "gdr2_scan.h"

namespace gdr2 {

namespace {

template <int NS> constexpr int kSub = NS <= 4 ? 16 : 8;   // tokens whose states are held

// Sum over lanes that differ in bits 2..5 (the 16 channels of a wave) of
// v[k][i], k the token of a group of four: lane (b5, b4) returns token
// k = 2 b5 + b4 in r[i].
template <int NS>
__device__ __forceinline__ void channel_sum(const float (&v)[4][NS], int lane, float (&r)[NS])
{
    const bool b5 = lane & 32, b4 = lane & 16;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const float w0 = (b5 ? v[2][i] : v[0][i]) + __shfl_xor(b5 ? v[0][i] : v[2][i], 32);
        const float w1 = (b5 ? v[3][i] : v[1][i]) + __shfl_xor(b5 ? v[1][i] : v[3][i], 32);
        float x = (b4 ? w1 : w0) + __shfl_xor(b4 ? w0 : w1, 16);
        x += __shfl_xor(x, 8);
        x += __shfl_xor(x, 4);
        r[i] = x;
    }
}

struct BackwardPtrs {
    float* parts;       // [ncb][rows][2][N]: dB, dC of one channel block
    float* sums;        // [slots][C (N + 2)]
    const float* lam;   // [slots][C][N] gradients entering each segment from behind, or NULL
};

template <typename T, int NS>
__global__ __launch_bounds__(256) void scan_backward_kernel(gdr2_scan_bwd_args p, Pieces seg, uint32_t ncb, uint32_t cb_per,
                                                            BackwardPtrs w)
{
    constexpr int NP = 4 * NS, SUB = kSub<NS>, NSUB = kScanChunk / SUB, NG = kScanChunk / 4;
    const gdr2_scan_args& a = p.f;
    __shared__ __align__(16) float s_b[kScanChunk][NP], s_c[kScanChunk][NP];
    __shared__ __align__(16) float s_red[2][4][SUB][NP];
    const uint32_t slot = blockIdx.x / ncb, cb = blockIdx.x - slot * ncb;
    const Piece q = uniform(piece_of(seg, slot));
    const ScanLane l = scan_lane(a, cb, cb_per);
    const int s = l.s, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t N = a.N, C = a.C, c = l.c;
    float* sums = w.sums + (int64_t)slot * C * (N + 2);
    float dA[NS] = {}, dskip = 0.f, dbias = 0.f;
    if (q.seq >= 0) {
        float A[NS], A2[NS], lam[NS];
        load_states<NS>(a.A + c * N, s, N, l.on, A);
#pragma unroll
        for (int i = 0; i < NS; ++i)
            A2[i] = A[i] * kLog2e;
        if (w.lam)
            load_states<NS>(w.lam + ((int64_t)slot * C + c) * N, s, N, l.on, lam);
        else
            load_states<NS>(p.dh_out + (q.seq * C + c) * N, s, N, l.on && p.dh_out, lam);
        const float bias = a.dt_bias && l.on ? a.dt_bias[c] : 0.f;
        const float skip = a.skip && l.on ? a.skip[c] : 0.f;
        const Pieces ckp{a.offsets, a.B, a.T, kScanLg};
        const int64_t ck0 = sequence_of(ckp, q.seq).first;
        const int64_t rows = a.offsets ? a.T : a.B * a.T;
        float* part = w.parts + (int64_t)cb * rows * 2 * N;
        const int64_t t0 = q.index << seg.lg;
        const int64_t t1 = min(q.len, t0 + ((int64_t)1 << seg.lg));
        for (int64_t t = t0 + ((t1 - t0 - 1) >> kScanLg << kScanLg); t1 > t0 && t >= t0; t -= kScanChunk) {
            __syncthreads();
            const int left = (int)min(t1 - t, (int64_t)kScanChunk);
            Staged<T, NP> rb(a.b_stride, l.j, (int)N), rc(a.c_stride, l.j, (int)N);
            rb.load(a.Bt, q.row0 + t, a.b_stride, left);
            rc.load(a.Ct, q.row0 + t, a.c_stride, left);
            rb.store(s_b);
            rc.store(s_c);
            float xs[NG], raws[NG], ds[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const int64_t mt = t + 4 * g + s, row = q.row0 + mt;
                xs[g] = raws[g] = ds[g] = 0.f;
                if (l.on && mt < t1) {
                    xs[g] = to_f32(((const T*)a.x)[row * a.x_stride + c]);
                    raws[g] = to_f32(((const T*)a.dt)[row * a.dt_stride + c]) + bias;
                    ds[g] = a.flags & GDR2_SCAN_SOFTPLUS ? softplus_f(raws[g]) : raws[g];
                }
            }
            __syncthreads();
            // the states before every SUB tokens
            float hs[NSUB][NS];
            load_states<NS>(a.h_chunks + ((ck0 + (t >> kScanLg)) * C + c) * N, s, N, l.on, hs[0]);
#pragma unroll
            for (int b = 1; b < NSUB; ++b) {
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    hs[b][i] = hs[b - 1][i];
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const int tt = (b - 1) * SUB + k;
                    const float dk = quad_bcast_k(ds[tt / 4], tt % 4);
                    const float uk = quad_bcast_k(ds[tt / 4] * xs[tt / 4], tt % 4);
#pragma unroll
                    for (int i = 0; i < NS; ++i)
                        hs[b][i] = fmaf(fast_exp2(dk * A2[i]), hs[b][i], uk * s_b[tt][s * NS + i]);
                }
            }
#pragma unroll
            for (int b = NSUB - 1; b >= 0; --b) {
                float av[SUB][NS], hv[SUB + 1][NS];
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    hv[0][i] = hs[b][i];
#pragma unroll
                for (int k = 0; k < SUB; ++k) {
                    const int tt = b * SUB + k;
                    const float dk = quad_bcast_k(ds[tt / 4], tt % 4);
                    const float uk = quad_bcast_k(ds[tt / 4] * xs[tt / 4], tt % 4);
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        av[k][i] = fast_exp2(dk * A2[i]);
                        hv[k + 1][i] = fmaf(av[k][i], hv[k][i], uk * s_b[tt][s * NS + i]);
                    }
                }
#pragma unroll
                for (int g = SUB / 4 - 1; g >= 0; --g) {
                    const int gg = b * (SUB / 4) + g;           // group within the chunk
                    const int64_t mt = t + 4 * gg + s, row = q.row0 + mt;
                    const bool in = l.on && mt < t1;
                    const float x = xs[gg], d = ds[gg], u = x * d;
                    float dy = in ? to_f32(((const T*)p.dy)[row * C + c]) : 0.f, z = 0.f, dv = dy;
                    if (a.z && in) {
                        z = to_f32(((const T*)a.z)[row * a.z_stride + c]);
                        dv = dy * silu_f(z);
                    }
                    float pu[4], pa[4], pv[4], vb[4][NS], vc[4][NS];
#pragma unroll
                    for (int k = 3; k >= 0; --k) {
                        const int tt = 4 * gg + k, kk = 4 * g + k;
                        const float dk = quad_bcast_k(d, k), uk = quad_bcast_k(u, k), dvk = quad_bcast_k(dv, k);
                        pu[k] = pa[k] = pv[k] = 0.f;
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            const float bn = s_b[tt][s * NS + i], cn = s_c[tt][s * NS + i];
                            const float gr = fmaf(cn, dvk, lam[i]);
                            vc[k][i] = dvk * hv[kk + 1][i];
                            vb[k][i] = gr * uk;
                            pu[k] = fmaf(gr, bn, pu[k]);
                            pv[k] = fmaf(cn, hv[kk + 1][i], pv[k]);
                            lam[i] = gr * av[kk][i];
                            const float qq = lam[i] * hv[kk][i];
                            pa[k] = fmaf(qq, A[i], pa[k]);
                            dA[i] = fmaf(qq, dk, dA[i]);
                        }
                    }
                    const float du = quad_sum_transposed(pu, s), qa = quad_sum_transposed(pa, s);
                    float dd = fmaf(x, du, qa);
                    if (a.flags & GDR2_SCAN_SOFTPLUS)
                        dd *= sigmoid_f(raws[gg]);
                    if (a.z) {
                        const float v = fmaf(skip, x, quad_sum_transposed(pv, s));
                        if (in)
                            ((T*)p.dz)[row * C + c] = from_f32<T>(dy * v * silu_slope_f(z));
                    }
                    if (in) {
                        ((T*)p.dx)[row * C + c] = from_f32<T>(fmaf(d, du, skip * dv));
                        ((T*)p.ddt)[row * C + c] = from_f32<T>(dd);
                        dskip = fmaf(dv, x, dskip);
                        dbias += dd;
                    }
                    float rb[NS], rc[NS];
                    channel_sum<NS>(vb, lane, rb);
                    channel_sum<NS>(vc, lane, rc);
                    if ((lane & 12) == 0) {
                        const int kr = 4 * g + (lane >> 4);
#pragma unroll
                        for (int i = 0; i < NS; ++i) {
                            s_red[0][wave][kr][s * NS + i] = rb[i];
                            s_red[1][wave][kr][s * NS + i] = rc[i];
                        }
                    }
                }
                __syncthreads();
                for (int e = threadIdx.x; e < 2 * SUB * NP; e += 256) {
                    const int which = e / (SUB * NP), r = e / NP % SUB, n = e % NP;
                    const int64_t mt = t + b * SUB + r;
                    if (mt < t1 && n < N)
                        part[((q.row0 + mt) * 2 + which) * N + n] = (s_red[which][0][r][n] + s_red[which][1][r][n]) +
                                                                     (s_red[which][2][r][n] + s_red[which][3][r][n]);
                }
                __syncthreads();
            }
        }
        if (p.dh0 && q.index == 0)
            store_states<NS>(p.dh0 + (q.seq * C + c) * N, s, N, l.on, lam);
    }
    store_states<NS>(sums + c * N, s, N, l.on, dA);
    dskip += dpp_quad_xor<1>(dskip);
    dskip += dpp_quad_xor<2>(dskip);
    dbias += dpp_quad_xor<1>(dbias);
    dbias += dpp_quad_xor<2>(dbias);
    if (l.on && s == 0) {
        sums[C * N + c] = dskip;
        sums[C * (N + 1) + c] = dbias;
    }
}

// Per segment but the first of its sequence: the gradient of its start state
// when none enters from behind, and sum d.
template <typename T, int NS>
__global__ __launch_bounds__(256) void scan_backward_span_kernel(gdr2_scan_bwd_args p, Pieces seg, uint32_t ncb,
                                                                 uint32_t cb_per, float* states, float* sums)
{
    constexpr int NP = 4 * NS;
    const gdr2_scan_args& a = p.f;
    __shared__ __align__(16) float s_c[kScanChunk][NP];
    const uint32_t slot = blockIdx.x / ncb;
    const Piece q = uniform(piece_of(seg, slot));
    if (q.seq < 0 || q.index == 0)
        return;
    const ScanLane l = scan_lane(a, blockIdx.x - slot * ncb, cb_per);
    const int s = l.s;
    const int64_t N = a.N, C = a.C, c = l.c;
    float A2[NS], lam[NS] = {}, sum = 0.f;
    load_states<NS>(a.A + c * N, s, N, l.on, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] *= kLog2e;
    const float bias = a.dt_bias && l.on ? a.dt_bias[c] : 0.f;
    const int64_t t0 = q.index << seg.lg;
    const int64_t t1 = min(q.len, t0 + ((int64_t)1 << seg.lg));
    for (int64_t t = t0 + ((t1 - t0 - 1) >> kScanLg << kScanLg); t >= t0; t -= kScanChunk) {
        __syncthreads();
        const int left = (int)min(t1 - t, (int64_t)kScanChunk);
        Staged<T, NP> rc(a.c_stride, l.j, (int)N);
        rc.load(a.Ct, q.row0 + t, a.c_stride, left);
        rc.store(s_c);
        __syncthreads();
#pragma unroll 1
        for (int tt = kScanChunk - 4; tt >= 0; tt -= 4) {
            const int64_t mt = t + tt + s, row = q.row0 + mt;
            float d = 0.f, dv = 0.f;
            if (l.on && mt < t1) {
                const float raw = to_f32(((const T*)a.dt)[row * a.dt_stride + c]) + bias;
                d = a.flags & GDR2_SCAN_SOFTPLUS ? softplus_f(raw) : raw;
                dv = to_f32(((const T*)p.dy)[row * C + c]);
                if (a.z)
                    dv *= silu_f(to_f32(((const T*)a.z)[row * a.z_stride + c]));
            }
            sum += d;
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const float dk = quad_bcast_k(d, k), dvk = quad_bcast_k(dv, k);
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    lam[i] = fmaf(s_c[tt + k][s * NS + i], dvk, lam[i]) * fast_exp2(dk * A2[i]);
            }
        }
    }
    sum += dpp_quad_xor<1>(sum);
    sum += dpp_quad_xor<2>(sum);
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
    const float A2 = a.A[cn] * kLog2e;
    float lam = p.dh_out ? p.dh_out[id] : 0.f;
    const int64_t nseg = max((int64_t)1, (q.len + ((int64_t)1 << seg.lg) - 1) >> seg.lg);
    for (int64_t i = nseg - 1; i >= 0; --i) {
        float* at = states + (q.first + i) * per + cn;
        float next = 0.f;
        if (i > 0)
            next = fmaf(fast_exp2(A2 * sums[(q.first + i) * a.C + c]), lam, *at);
        *at = lam;
        lam = next;
    }
}

// dB and dC: the channel blocks' partial sums of each row, in block order.
template <typename T>
__global__ __launch_bounds__(256) void scan_rows_sum_kernel(gdr2_scan_bwd_args p, const float* parts, int64_t rows, int64_t cb_per)
{
    const gdr2_scan_args& a = p.f;
    const int64_t N = a.N, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= rows * a.G * N)
        return;
    const int64_t row = id / (a.G * N), jn = id - row * a.G * N, j = jn / N, n = jn - j * N;
    if (a.offsets) {
        // rows of no sequence: before the first or behind the last
        const Pieces pc{a.offsets, a.B, a.T, 0};
        if (row < clamp_offset(pc, 0) || row >= clamp_offset(pc, a.B))
            return;
    }
    const float* at = parts + ((j * cb_per * rows + row) * 2) * N + n;
    float db = 0.f, dc = 0.f;
    for (int64_t i = 0; i < cb_per; ++i) {
        db += at[i * rows * 2 * N];
        dc += at[i * rows * 2 * N + N];
    }
    ((T*)p.dBt)[id] = from_f32<T>(db);
    ((T*)p.dCt)[id] = from_f32<T>(dc);
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
    w.lam = w.sums + al((size_t)slots * a.C * (a.N + 2) * 4);
    w.span = w.lam + (pl.split ? al((size_t)slots * a.C * a.N * 4) : 0);
    w.total = w.span + (pl.split ? (size_t)slots * a.C * 4 : 0);
    return w;
}

template <typename T, int NS>
hipError_t backward_t(const gdr2_scan_bwd_args& p, hipStream_t stream)
{
    const gdr2_scan_args& a = p.f;
    const ScanPlan pl = scan_plan(a, true);
    const BackwardWork w = backward_work(p, pl);
    char* ws = (char*)p.workspace;
    const dim3 grid((unsigned)(pl.seg.slots() * pl.ncb));
    const int64_t rows = a.offsets ? a.T : a.B * a.T;
    BackwardPtrs ptr{(float*)(ws + w.parts), (float*)(ws + w.sums), nullptr};
    hipError_t e;
    if (a.B == 0)      // no rows: zeros are all there is to write
        return launch_column_sum(ptr.sums, 0, {p.dA, a.C * a.N}, {p.dskip, a.C}, {p.ddt_bias, a.C}, stream);
    if (pl.split) {
        float* lam = (float*)(ws + w.lam);
        float* span = (float*)(ws + w.span);
        hipLaunchKernelGGL((scan_backward_span_kernel<T, NS>), grid, dim3(256), 0, stream, p, pl.seg, (uint32_t)pl.ncb,
                           (uint32_t)pl.cb_per, lam, span);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        hipLaunchKernelGGL(scan_backward_fold_kernel, dim3((unsigned)ceil_div(a.B * a.C * a.N, 256)), dim3(256), 0, stream, p,
                           pl.seg, lam, span);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
        ptr.lam = lam;
    }
    hipLaunchKernelGGL((scan_backward_kernel<T, NS>), grid, dim3(256), 0, stream, p, pl.seg, (uint32_t)pl.ncb,
                       (uint32_t)pl.cb_per, ptr);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    if (rows > 0) {
        hipLaunchKernelGGL((scan_rows_sum_kernel<T>), dim3((unsigned)ceil_div(rows * a.G * a.N, 256)), dim3(256), 0, stream, p,
                           ptr.parts, rows, pl.cb_per);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    return launch_column_sum(ptr.sums, pl.seg.slots(), {p.dA, a.C * a.N}, {p.dskip, a.C}, {p.ddt_bias, a.C}, stream);
}

}  // namespace

size_t scan_backward_workspace_bytes(const gdr2_scan_bwd_args& p) { return backward_work(p, scan_plan(p.f, true)).total; }

hipError_t launch_scan_backward(const gdr2_scan_bwd_args& p, hipStream_t stream)
{
    const gdr2_scan_args& a = p.f;
    const bool bf = a.dtype == GDR2_BF16;
    if (a.N <= 8)
        return bf ? backward_t<bf16, 2>(p, stream) : backward_t<float, 2>(p, stream);
    if (a.N <= 16)
        return bf ? backward_t<bf16, 4>(p, stream) : backward_t<float, 4>(p, stream);
    return bf ? backward_t<bf16, 8>(p, stream) : backward_t<float, 8>(p, stream);
}

}  // namespace gdr2
