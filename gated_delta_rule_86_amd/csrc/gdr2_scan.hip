// gdr2_scan.hip -- the selective state space scan, forwards: prompts (one
// pass, or segments of long sequences in parallel) and single tokens.
//
//   h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,   v_t = C_t . h_t + skip x_t,
//   y_t = v_t silu(z_t)
//
// Per (token, channel, state): one multiply for the exponent, one exp2, and
// three multiply-adds.  At 16 states that arithmetic, not the 8 bytes a
// channel moves per token, bounds a prompt.
//
// Segments: h is linear in its start, so over a segment h_end = P h_start + E
// with P = exp(A sum d) and E the end state from zero.  A span pass forms
// (sum d, E) of every segment but a sequence's last, a fold chains the
// segments' start states, and the main pass runs them all at once.
#include "gdr2_scan.h"

namespace gdr2 {

namespace {

// The step of a token.
__device__ __forceinline__ float step_of(float dt, float bias, int flags)
{
    const float raw = dt + bias;
    return flags & GDR2_SCAN_SOFTPLUS ? softplus_f(raw) : raw;
}

// Both passes walk a segment chunk by chunk.  The rows of the next chunk are
// requested before the current one is computed (there is about one wave per
// SIMD, so nothing else hides their latency), and B and C alternate between
// two LDS buffers, so a chunk costs one barrier.
template <typename T, int NS, bool GATE>
__global__ __launch_bounds__(256) void scan_forward_kernel(gdr2_scan_args a, Pieces seg, uint32_t ncb, uint32_t cb_per,
                                                           const float* starts)
{
    constexpr int NP = 4 * NS;
    __shared__ __align__(16) float s_b[2][kScanChunk][NP], s_c[2][kScanChunk][NP];
    const uint32_t slot = blockIdx.x / ncb;
    const Piece q = uniform(piece_of(seg, slot));
    if (q.seq < 0)
        return;
    const ScanLane l = scan_lane(a, blockIdx.x - slot * ncb, cb_per);
    const int s = l.s, N = (int)a.N;
    const int64_t c = l.c, j = uniform(l.j);
    float A2[NS], h[NS];
    load_states<NS>(a.A + c * N, s, N, l.on, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] *= kLog2e;
    if (starts)
        load_states<NS>(starts + ((int64_t)slot * a.C + c) * N, s, N, l.on, h);
    else
        load_states<NS>(a.h0 + (q.seq * a.C + c) * N, s, N, l.on && a.h0, h);
    const float bias = a.dt_bias && l.on ? a.dt_bias[c] : 0.f;
    const float skip = a.skip && l.on ? a.skip[c] : 0.f;
    const Pieces ckp{a.offsets, a.B, a.T, kScanLg};
    const int64_t ck0 = uniform(sequence_of(ckp, q.seq).first);

    const int64_t t0 = q.index << seg.lg;
    const int64_t t1 = min(q.len, t0 + ((int64_t)1 << seg.lg));
    const TokenRows<T> xs(a.x_stride, c, s, l.on), ts(a.dt_stride, c, s, l.on), zs(a.z_stride, c, s, l.on), ys(a.C, c, s, l.on);
    uint32_t rx[kGroups], rt[kGroups], rz[kGroups] = {};
    Staged<T, NP> rb(a.b_stride, j, N), rc(a.c_stride, j, N);
    auto fetch = [&](int64_t t) {
        const int left = (int)min(t1 - t, (int64_t)kScanChunk);
        rb.load(a.Bt, q.row0 + t, a.b_stride, left);
        rc.load(a.Ct, q.row0 + t, a.c_stride, left);
        ts.load(a.dt, q.row0 + t, a.dt_stride, left, rt);
        xs.load(a.x, q.row0 + t, a.x_stride, left, rx);
        if constexpr (GATE)
            zs.load(a.z, q.row0 + t, a.z_stride, left, rz);
    };
    if (t0 < t1)
        fetch(t0);
    int buf = 0;
    for (int64_t t = t0; t < t1; t += kScanChunk, buf ^= 1) {
        const int left = (int)min(t1 - t, (int64_t)kScanChunk);
        float x[kGroups], pre[kGroups], d[kGroups], z[kGroups];
        rb.store(s_b[buf]);
        rc.store(s_c[buf]);
        chunk_steps<T>(rt, bias, a.flags, s, left, pre, d);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            x[g] = raw_f32<T>(rx[g]);
            z[g] = raw_f32<T>(rz[g]);
        }
        if (t + kScanChunk < t1)
            fetch(t + kScanChunk);
        if (a.h_chunks)
            store_states<NS>(a.h_chunks + ((ck0 + (t >> kScanLg)) * a.C + c) * N, s, N, l.on, h);
        __syncthreads();
        const auto yb = chunk_buffer<T>(a.y, q.row0 + t, a.C, left);
        Quad<NS> bq[2], cq[2];
        bq[0].template read<NP>(s_b[buf], 0, s);
        cq[0].template read<NP>(s_c[buf], 0, s);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            if (g + 1 < kGroups) {
                bq[(g + 1) & 1].template read<NP>(s_b[buf], 4 * g + 4, s);
                cq[(g + 1) & 1].template read<NP>(s_c[buf], 4 * g + 4, s);
            }
            __builtin_amdgcn_sched_barrier(0);
            const float u = d[g] * x[g];
            float p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float dk = quad_bcast_k(d[g], k), uk = quad_bcast_k(u, k);
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[i] = fmaf(fast_exp2(dk * A2[i]), h[i], uk * bq[g & 1].v[k][i]);
                    p[k] = i == 0 ? cq[g & 1].v[k][0] * h[0] : fmaf(cq[g & 1].v[k][i], h[i], p[k]);
                }
            }
            float y = fmaf(skip, x[g], quad_sum_transposed(p, s));
            if constexpr (GATE)
                y *= silu_f(z[g]);
            buffer_put<T>(yb, ys.off[g], from_f32<T>(y));
        }
    }
    if (a.h_out && t1 == q.len)
        store_states<NS>(a.h_out + (q.seq * a.C + c) * N, s, N, l.on, h);
}

// (sum d, E) of every segment but the last of its sequence: whole segments.
template <typename T, int NS>
__global__ __launch_bounds__(256) void scan_span_kernel(gdr2_scan_args a, Pieces seg, uint32_t ncb, uint32_t cb_per,
                                                        float* states, float* sums)
{
    constexpr int NP = 4 * NS;
    __shared__ __align__(16) float s_b[2][kScanChunk][NP];
    const uint32_t slot = blockIdx.x / ncb;
    const Piece q = uniform(piece_of(seg, slot));
    const int64_t t0 = q.index << seg.lg, t1 = t0 + ((int64_t)1 << seg.lg);
    if (q.seq < 0 || t1 >= q.len)
        return;
    const ScanLane l = scan_lane(a, blockIdx.x - slot * ncb, cb_per);
    const int s = l.s, N = (int)a.N;
    const int64_t c = l.c, j = uniform(l.j);
    float A2[NS], h[NS] = {}, sum = 0.f;
    load_states<NS>(a.A + c * N, s, N, l.on, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i)
        A2[i] *= kLog2e;
    const float bias = a.dt_bias && l.on ? a.dt_bias[c] : 0.f;
    const TokenRows<T> xs(a.x_stride, c, s, l.on), ts(a.dt_stride, c, s, l.on);
    uint32_t rx[kGroups], rt[kGroups];
    Staged<T, NP> rb(a.b_stride, j, N);
    auto fetch = [&](int64_t t) {
        rb.load(a.Bt, q.row0 + t, a.b_stride, kScanChunk);
        ts.load(a.dt, q.row0 + t, a.dt_stride, kScanChunk, rt);
        xs.load(a.x, q.row0 + t, a.x_stride, kScanChunk, rx);
    };
    fetch(t0);
    int buf = 0;
    for (int64_t t = t0; t < t1; t += kScanChunk, buf ^= 1) {
        float u[kGroups], pre[kGroups], d[kGroups];
        rb.store(s_b[buf]);
        chunk_steps<T>(rt, bias, a.flags, s, kScanChunk, pre, d);
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            u[g] = d[g] * raw_f32<T>(rx[g]);
        if (t + kScanChunk < t1)
            fetch(t + kScanChunk);
        __syncthreads();
        Quad<NS> bq[2];
        bq[0].template read<NP>(s_b[buf], 0, s);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            if (g + 1 < kGroups)
                bq[(g + 1) & 1].template read<NP>(s_b[buf], 4 * g + 4, s);
            __builtin_amdgcn_sched_barrier(0);
            sum += d[g];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float dk = quad_bcast_k(d[g], k), uk = quad_bcast_k(u[g], k);
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    h[i] = fmaf(fast_exp2(dk * A2[i]), h[i], uk * bq[g & 1].v[k][i]);
            }
        }
    }
    sum += dpp_quad_xor<1>(sum);
    sum += dpp_quad_xor<2>(sum);
    store_states<NS>(states + ((int64_t)slot * a.C + c) * N, s, N, l.on, h);
    if (l.on && s == 0)
        sums[(int64_t)slot * a.C + c] = sum;
}

// Start states of a sequence's segments, written over the E of each.  One
// thread per (sequence, channel, state).
__global__ __launch_bounds__(256) void scan_fold_kernel(gdr2_scan_args a, Pieces seg, float* states, const float* sums)
{
    const int64_t per = a.C * a.N;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.B * per)
        return;
    const int64_t seq = id / per, cn = id - seq * per, c = cn / a.N;
    const Piece q = sequence_of(seg, seq);
    const float A2 = a.A[cn] * kLog2e;
    float h = a.h0 ? a.h0[id] : 0.f;
    const int64_t nseg = max((int64_t)1, (q.len + ((int64_t)1 << seg.lg) - 1) >> seg.lg);
    for (int64_t i = 0; i < nseg; ++i) {
        float* at = states + (q.first + i) * per + cn;
        float next = 0.f;
        if (i + 1 < nseg)
            next = fmaf(fast_exp2(A2 * sums[(q.first + i) * a.C + c]), h, *at);
        *at = h;
        h = next;
    }
}

// One token.  LPC lanes per channel, four states each.
template <typename T, int LPC>
__global__ __launch_bounds__(256) void scan_step_kernel(gdr2_scan_step_args p)
{
    const gdr2_scan_args& a = p.s;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t bc = item / LPC;
    const int s = threadIdx.x % LPC;
    const bool on = bc < a.B * a.C;
    const int64_t b = on ? bc / a.C : 0, c = on ? bc - b * a.C : 0;
    const int64_t N = a.N, j = c / (a.C / a.G);
    float* st = p.state + (b * a.C + c) * N;
    float h[4], A[4], Bv[4], Cv[4];
    load_states<4>(st, s, N, on, h);
    load_states<4>(a.A + c * N, s, N, on, A);
    const T* Bt = (const T*)a.Bt + b * a.b_stride + j * N;
    const T* Ct = (const T*)a.Ct + b * a.c_stride + j * N;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = on && s * 4 + i < N;
        Bv[i] = in ? to_f32(Bt[s * 4 + i]) : 0.f;
        Cv[i] = in ? to_f32(Ct[s * 4 + i]) : 0.f;
    }
    const float x = on ? to_f32(((const T*)a.x)[b * a.x_stride + c]) : 0.f;
    const float d = on ? step_of(to_f32(((const T*)a.dt)[b * a.dt_stride + c]), a.dt_bias ? a.dt_bias[c] : 0.f, a.flags) : 0.f;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(fast_exp2(d * (A[i] * kLog2e)), h[i], d * x * Bv[i]);
        y = fmaf(Cv[i], h[i], y);
    }
    store_states<4>(st, s, N, on, h);
#pragma unroll
    for (int off = LPC / 2; off >= 1; off >>= 1)
        y += __shfl_xor(y, off);
    if (on && s == 0) {
        y = fmaf(a.skip ? a.skip[c] : 0.f, x, y);
        if (a.z)
            y *= silu_f(to_f32(((const T*)a.z)[b * a.z_stride + c]));
        ((T*)a.y)[b * a.C + c] = from_f32<T>(y);
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

template <typename T, int NS>
hipError_t forward_t(const gdr2_scan_args& a, hipStream_t stream)
{
    const ScanPlan p = scan_plan(a, false);
    const ForwardWork w = forward_work(a, p);
    const dim3 grid((unsigned)(p.seg.slots() * p.ncb));
    float* states = nullptr;
    if (p.split) {
        states = (float*)((char*)a.workspace + w.states);
        float* sums = (float*)((char*)a.workspace + w.sums);
        hipLaunchKernelGGL((scan_span_kernel<T, NS>), grid, dim3(256), 0, stream, a, p.seg, (uint32_t)p.ncb, (uint32_t)p.cb_per,
                           states, sums);
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
        hipLaunchKernelGGL((scan_forward_kernel<T, NS, true>), grid, dim3(256), 0, stream, a, p.seg, (uint32_t)p.ncb,
                           (uint32_t)p.cb_per, states);
    else
        hipLaunchKernelGGL((scan_forward_kernel<T, NS, false>), grid, dim3(256), 0, stream, a, p.seg, (uint32_t)p.ncb,
                           (uint32_t)p.cb_per, states);
    return hipGetLastError();
}

template <typename T, int LPC>
hipError_t step_t(const gdr2_scan_step_args& a, hipStream_t stream)
{
    hipLaunchKernelGGL((scan_step_kernel<T, LPC>), dim3((unsigned)ceil_div(a.s.B * a.s.C * LPC, 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t step_n(const gdr2_scan_step_args& a, hipStream_t stream)
{
    if (a.s.N <= 4)
        return step_t<T, 1>(a, stream);
    if (a.s.N <= 8)
        return step_t<T, 2>(a, stream);
    return a.s.N <= 16 ? step_t<T, 4>(a, stream) : step_t<T, 8>(a, stream);
}

}  // namespace

// One segment per sequence unless that leaves compute units without a
// workgroup; then the shortest power of two of chunks that gives about
// that many, at least four chunks.
ScanPlan scan_plan(const gdr2_scan_args& a, bool backward)
{
    ScanPlan p;
    p.cb_per = ceil_div(a.C / a.G, kScanCols);
    p.ncb = p.cb_per * a.G;
    const int64_t want = (int64_t)device_cu_count();
    int whole = kScanLg;                      // a segment that holds any sequence
    while (((int64_t)1 << whole) < a.T)
        ++whole;
    int lg = whole;
    if (a.algo == GDR2_ALGO_SEGMENTED)
        lg = min(whole, kScanLg + 1);
    else if (a.algo == GDR2_ALGO_AUTO)
        while (lg > kScanLg + 2 && Pieces{a.offsets, a.B, a.T, lg}.slots() * p.ncb < want)
            --lg;
    p.seg = Pieces{a.offsets, a.B, a.T, lg};
    p.split = lg < whole;
    return p;
}

int64_t scan_launch_groups(const gdr2_scan_args& a)
{
    const ScanPlan p = scan_plan(a, true);
    int64_t n;
    if (__builtin_mul_overflow(p.seg.slots(), p.ncb, &n))
        return kMaxGroups;
    return max(n, ceil_div(a.B * a.C * max((int64_t)8, a.N), 256));
}

size_t scan_workspace_bytes(const gdr2_scan_args& a) { return forward_work(a, scan_plan(a, false)).total; }

hipError_t launch_scan_forward(const gdr2_scan_args& a, hipStream_t stream)
{
    const bool bf = a.dtype == GDR2_BF16;
    if (a.N <= 8)
        return bf ? forward_t<bf16, 2>(a, stream) : forward_t<float, 2>(a, stream);
    if (a.N <= 16)
        return bf ? forward_t<bf16, 4>(a, stream) : forward_t<float, 4>(a, stream);
    return bf ? forward_t<bf16, 8>(a, stream) : forward_t<float, 8>(a, stream);
}

hipError_t launch_scan_step(const gdr2_scan_step_args& a, hipStream_t stream)
{
    return a.s.dtype == GDR2_BF16 ? step_n<bf16>(a, stream) : step_n<float>(a, stream);
}

}  // namespace gdr2
