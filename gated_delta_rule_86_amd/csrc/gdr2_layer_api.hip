// gdr2_layer_api.hip -- the C ABI of the layer operators (convolution, scan,
// norm): host-side validation and dispatch.  Every check runs before any
// launch; a failed check launches nothing and leaves the outputs untouched.
#include "gdr2_checks.h"
#include "gdr2_layer.h"

namespace {

using namespace gdr2;

// ---- convolution -----------------------------------------------------------

// Sizes and modes common to the convolution's entry points.
gdr2_status check_conv(int64_t B, int64_t T, int64_t C, int64_t x_stride, int32_t width, int32_t dtype, int32_t act,
                       int32_t reserved)
{
    if (B < 0 || T < 0)
        return set_error(GDR2_ERR_INVALID_ARG, "sizes must be >= 0");
    if (C <= 0)
        return set_error(GDR2_ERR_INVALID_ARG, "C must be positive (got %lld)", (long long)C);
    GDR2_TRY(check_dtype(dtype, reserved));
    if (act != GDR2_ACT_NONE && act != GDR2_ACT_SILU)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown activation %d", act);
    if (width < 2 || width > 4)
        return set_error(GDR2_ERR_UNSUPPORTED, "supported widths: 2, 3, 4 (got %d)", width);
    GDR2_TRY(check_stride("x_stride", x_stride, C));
    return B > ((int64_t)1 << 40) || T > ((int64_t)1 << 40) ? too_many() : GDR2_OK;
}

gdr2_status validate(const gdr2_conv_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_conv(a->B, a->T, a->C, a->x_stride, a->width, a->dtype, a->act, a->reserved));
    if (gdr2::conv_forward_groups(*a) >= gdr2::kMaxGroups)
        return too_many();
    const int64_t e = elt(a->dtype), rows = a->B == 0 ? 0 : a->offsets ? a->T : mul(a->B, a->T);
    const int64_t st = mul(mul(a->B, a->width - 1), a->C);
    const Buf b[] = {
        rows_in("x", a->x, rows, a->C, a->x_stride, e),
        dense("weight", a->weight, mul(a->C, a->width), 4, false),
        dense("bias", a->bias, a->C, 4, false, false),
        dense("state0", a->state0, st, e, false, false),
        {"offsets", a->offsets, mul(a->B + 1, 8), 8, false, false},
        dense("y", a->y, mul(rows, a->C), e, true),
        dense("state_out", a->state_out, st, e, true, false),
    };
    return check_bufs(b, 7, "state_out", "state0");
}

gdr2_status validate(const gdr2_conv_step_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_conv(a->N, 1, a->C, a->x_stride, a->width, a->dtype, a->act, a->reserved));
    if (gdr2::conv_step_groups(*a) >= gdr2::kMaxGroups)
        return too_many();
    const int64_t e = elt(a->dtype);
    const Buf b[] = {
        rows_in("x", a->x, a->N, a->C, a->x_stride, e),
        dense("weight", a->weight, mul(a->C, a->width), 4, false),
        dense("bias", a->bias, a->C, 4, false, false),
        dense("state", a->state, mul(mul(a->N, a->width - 1), a->C), e, true),
        dense("y", a->y, mul(a->N, a->C), e, true),
    };
    return check_bufs(b, 5);
}

gdr2_status check_sizes(const gdr2_conv_bwd_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_conv(a->B, a->T, a->C, a->x_stride, a->width, a->dtype, a->act, a->reserved));
    return gdr2::conv_backward_groups(*a) >= gdr2::kMaxGroups ? too_many() : GDR2_OK;
}

gdr2_status validate(const gdr2_conv_bwd_args* a)
{
    GDR2_TRY(check_sizes(a));
    const int64_t e = elt(a->dtype), rows = a->B == 0 ? 0 : a->offsets ? a->T : mul(a->B, a->T);
    const int64_t st = mul(mul(a->B, a->width - 1), a->C);
    const size_t need = gdr2::conv_backward_workspace_bytes(*a);
    GDR2_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const Buf b[] = {
        rows_in("x", a->x, rows, a->C, a->x_stride, e),
        dense("weight", a->weight, mul(a->C, a->width), 4, false),
        dense("bias", a->bias, a->C, 4, false, false),
        dense("state0", a->state0, st, e, false, false),
        {"offsets", a->offsets, mul(a->B + 1, 8), 8, false, false},
        dense("dy", a->dy, mul(rows, a->C), e, false),
        dense("dstate", a->dstate, st, e, false, false),
        dense("dx", a->dx, mul(rows, a->C), e, true),
        dense("dweight", a->dweight, mul(a->C, a->width), 4, true),
        dense("dbias", a->dbias, a->C, 4, true, false),
        dense("dstate0", a->dstate0, st, e, true, false),
        dense("workspace", a->workspace, (int64_t)need, 1, true),
    };
    return check_bufs(b, 12);
}

// ---- scan ------------------------------------------------------------------

gdr2_status check_scan(const gdr2_scan_args& a, gdr2::ScanCall call)
{
    if (a.B < 0 || a.T < 0)
        return set_error(GDR2_ERR_INVALID_ARG, "B, T must be >= 0");
    if (a.C <= 0 || a.N <= 0 || a.G <= 0)
        return set_error(GDR2_ERR_INVALID_ARG, "C, N, G must be positive (got %lld, %lld, %lld)", (long long)a.C,
                         (long long)a.N, (long long)a.G);
    GDR2_TRY(check_dtype(a.dtype, a.reserved));
    if (a.C % a.G)
        return set_error(GDR2_ERR_INVALID_ARG, "G = %lld must divide C = %lld", (long long)a.G, (long long)a.C);
    if (a.flags & ~GDR2_SCAN_SOFTPLUS)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown flags 0x%x", a.flags);
    if (a.algo != GDR2_ALGO_AUTO && a.algo != GDR2_ALGO_STAGED && a.algo != GDR2_ALGO_SEGMENTED)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown algo %d", a.algo);
    if (a.N > 32)
        return set_error(GDR2_ERR_UNSUPPORTED, "supported state sizes: 1 to 32 (got %lld)", (long long)a.N);
    const int64_t most = call == gdr2::ScanCall::Step ? kMaxStride : kScanMaxStride;
    GDR2_TRY(check_stride("x_stride", a.x_stride, a.C, most));
    GDR2_TRY(check_stride("dt_stride", a.dt_stride, a.C, most));
    if (a.z)
        GDR2_TRY(check_stride("z_stride", a.z_stride, a.C, most));
    GDR2_TRY(check_stride("b_stride", a.b_stride, a.G * a.N, most));
    GDR2_TRY(check_stride("c_stride", a.c_stride, a.G * a.N, most));
    const int64_t rows = a.offsets ? a.T : mul(a.B, a.T);
    if (a.B > ((int64_t)1 << 31) || a.T > ((int64_t)1 << 40) || rows > ((int64_t)1 << 40) ||
        gdr2::scan_launch_groups(a, call) >= gdr2::kMaxGroups)
        return too_many();
    return GDR2_OK;
}

int64_t scan_rows(const gdr2_scan_args& a) { return a.B == 0 ? 0 : a.offsets ? a.T : a.B * a.T; }

int64_t chunk_floats(const gdr2_scan_args& a)
{
    return mul(mul(gdr2_scan_chunk_count(a.B, a.T, a.offsets != nullptr), a.C), a.N);
}

// The inputs the forward and the backward share (11 buffers).
void scan_inputs(const gdr2_scan_args& a, Buf* b)
{
    const int64_t e = elt(a.dtype), rows = scan_rows(a);
    b[0] = rows_in("x", a.x, rows, a.C, a.x_stride, e);
    b[1] = rows_in("dt", a.dt, rows, a.C, a.dt_stride, e);
    b[2] = rows_in("Bt", a.Bt, rows, a.G * a.N, a.b_stride, e);
    b[3] = rows_in("Ct", a.Ct, rows, a.G * a.N, a.c_stride, e);
    b[4] = rows_in("z", a.z, rows, a.C, a.z_stride, e, false);
    b[5] = dense("A", a.A, mul(a.C, a.N), 4, false);
    b[6] = dense("skip", a.skip, a.C, 4, false, false);
    b[7] = dense("dt_bias", a.dt_bias, a.C, 4, false, false);
    b[8] = Buf{"offsets", a.offsets, mul(a.B + 1, 8), 8, false, false};
}

gdr2_status validate(const gdr2_scan_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_scan(*a, gdr2::ScanCall::Forward));
    const size_t need = gdr2::scan_workspace_bytes(*a);
    GDR2_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const int64_t st = mul(mul(a->B, a->C), a->N);
    Buf b[14];
    scan_inputs(*a, b);
    b[9] = dense("h0", a->h0, st, 4, false, false);
    b[10] = dense("y", a->y, mul(scan_rows(*a), a->C), elt(a->dtype), true);
    b[11] = dense("h_out", a->h_out, st, 4, true, false);
    b[12] = dense("h_chunks", a->h_chunks, chunk_floats(*a), 4, true, false);
    b[13] = dense("workspace", a->workspace, (int64_t)need, 1, true);
    return check_bufs(b, 14, "h_out", "h0");
}

gdr2_status validate(const gdr2_scan_step_args* p)
{
    if (!p)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    const gdr2_scan_args& a = p->s;
    if (a.T != 1 || a.offsets || a.h0 || a.h_out || a.h_chunks)
        return set_error(GDR2_ERR_INVALID_ARG, "a step has T = 1 and no offsets, h0, h_out or h_chunks");
    GDR2_TRY(check_scan(a, gdr2::ScanCall::Step));
    Buf b[11];
    scan_inputs(a, b);
    b[9] = dense("state", p->state, mul(mul(a.B, a.C), a.N), 4, true);
    b[10] = dense("y", a.y, mul(a.B, a.C), elt(a.dtype), true);
    return check_bufs(b, 11);
}

gdr2_status check_sizes(const gdr2_scan_bwd_args* p)
{
    if (!p)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    return check_scan(p->f, gdr2::ScanCall::Backward);
}

gdr2_status validate(const gdr2_scan_bwd_args* p)
{
    GDR2_TRY(check_sizes(p));
    const gdr2_scan_args& a = p->f;
    if (!a.z && p->dz)
        return set_error(GDR2_ERR_INVALID_ARG, "dz given without z");
    const size_t need = gdr2::scan_backward_workspace_bytes(*p);
    GDR2_TRY(check_workspace(p->workspace, p->workspace_bytes, need));
    const int64_t e = elt(a.dtype), rows = scan_rows(a), st = mul(mul(a.B, a.C), a.N);
    Buf b[22];
    scan_inputs(a, b);
    b[9] = dense("h_chunks", a.h_chunks, chunk_floats(a), 4, false);
    b[10] = dense("dy", p->dy, mul(rows, a.C), e, false);
    b[11] = dense("dh_out", p->dh_out, st, 4, false, false);
    b[12] = dense("dx", p->dx, mul(rows, a.C), e, true);
    b[13] = dense("ddt", p->ddt, mul(rows, a.C), e, true);
    b[14] = dense("dBt", p->dBt, mul(rows, a.G * a.N), e, true);
    b[15] = dense("dCt", p->dCt, mul(rows, a.G * a.N), e, true);
    b[16] = dense("dz", p->dz, mul(rows, a.C), e, true, a.z != nullptr);
    b[17] = dense("dA", p->dA, mul(a.C, a.N), 4, true);
    b[18] = dense("dskip", p->dskip, a.C, 4, true, false);
    b[19] = dense("ddt_bias", p->ddt_bias, a.C, 4, true, false);
    b[20] = dense("dh0", p->dh0, st, 4, true, false);
    b[21] = dense("workspace", p->workspace, (int64_t)need, 1, true);
    return check_bufs(b, 22, "dh0", "dh_out");
}

// ---- norm ------------------------------------------------------------------

gdr2_status check_norm(const gdr2_norm_args& a, bool backward)
{
    if (a.R < 0)
        return set_error(GDR2_ERR_INVALID_ARG, "R must be >= 0");
    if (a.C <= 0)
        return set_error(GDR2_ERR_INVALID_ARG, "C must be positive (got %lld)", (long long)a.C);
    GDR2_TRY(check_dtype(a.dtype, a.reserved));
    if (a.kind != GDR2_NORM_LAYER && a.kind != GDR2_NORM_RMS)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown kind %d", a.kind);
    if (!(a.eps >= 0.f) || std::isinf(a.eps))
        return set_error(GDR2_ERR_INVALID_ARG, "eps must be finite and >= 0");
    GDR2_TRY(check_stride("x_stride", a.x_stride, a.C));
    if (a.z)
        GDR2_TRY(check_stride("z_stride", a.z_stride, a.C));
    if (a.R >= ((int64_t)1 << 40) || gdr2::norm_launch_groups(a, backward) >= gdr2::kMaxGroups)
        return too_many();
    return GDR2_OK;
}

gdr2_status validate(const gdr2_norm_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_norm(*a, false));
    const int64_t e = elt(a->dtype);
    const Buf b[] = {
        rows_in("x", a->x, a->R, a->C, a->x_stride, e),
        rows_in("z", a->z, a->R, a->C, a->z_stride, e, false),
        dense("weight", a->weight, a->C, 4, false, false),
        dense("bias", a->bias, a->C, 4, false, false),
        dense("y", a->y, mul(a->R, a->C), e, true),
    };
    return check_bufs(b, 5);
}

gdr2_status check_sizes(const gdr2_norm_bwd_args* p)
{
    if (!p)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    return check_norm(p->f, true);
}

gdr2_status validate(const gdr2_norm_bwd_args* p)
{
    GDR2_TRY(check_sizes(p));
    const gdr2_norm_args& a = p->f;
    if (!a.z && p->dz)
        return set_error(GDR2_ERR_INVALID_ARG, "dz given without z");
    const size_t need = gdr2::norm_backward_workspace_bytes(*p);
    GDR2_TRY(check_workspace(p->workspace, p->workspace_bytes, need));
    const int64_t e = elt(a.dtype), n = mul(a.R, a.C);
    const Buf b[] = {
        rows_in("x", a.x, a.R, a.C, a.x_stride, e),
        rows_in("z", a.z, a.R, a.C, a.z_stride, e, false),
        dense("weight", a.weight, a.C, 4, false, false),
        dense("bias", a.bias, a.C, 4, false, false),
        dense("dy", p->dy, n, e, false),
        dense("dx", p->dx, n, e, true),
        dense("dz", p->dz, n, e, true, a.z != nullptr),
        dense("dweight", p->dweight, a.C, 4, true, false),
        dense("dbias", p->dbias, a.C, 4, true, false),
        dense("workspace", p->workspace, (int64_t)need, 1, true),
    };
    return check_bufs(b, 10);
}

}  // namespace

extern "C" {

gdr2_status gdr2_conv_forward(const gdr2_conv_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->B == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_conv_forward(*a, (hipStream_t)stream), (hipStream_t)stream, "convolution");
}

gdr2_status gdr2_conv_step(const gdr2_conv_step_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->N == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_conv_step(*a, (hipStream_t)stream), (hipStream_t)stream, "convolution step");
}

size_t gdr2_conv_backward_workspace_size(const gdr2_conv_bwd_args* a)
{
    return check_sizes(a) == GDR2_OK ? gdr2::conv_backward_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_conv_backward(const gdr2_conv_bwd_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    return hip_result(gdr2::launch_conv_backward(*a, (hipStream_t)stream), (hipStream_t)stream, "convolution backward");
}

int64_t gdr2_scan_chunk_count(int64_t B, int64_t T, int packed)
{
    if (B <= 0 || T < 0)
        return 0;
    return packed ? T / GDR2_SCAN_CHUNK + B : mul(B, T / GDR2_SCAN_CHUNK + (T % GDR2_SCAN_CHUNK != 0));
}

size_t gdr2_scan_workspace_size(const gdr2_scan_args* a)
{
    return a && check_scan(*a, gdr2::ScanCall::Forward) == GDR2_OK ? gdr2::scan_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_scan_forward(const gdr2_scan_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->B == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_scan_forward(*a, (hipStream_t)stream), (hipStream_t)stream, "scan");
}

gdr2_status gdr2_scan_step(const gdr2_scan_step_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->s.B == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_scan_step(*a, (hipStream_t)stream), (hipStream_t)stream, "scan step");
}

size_t gdr2_scan_backward_workspace_size(const gdr2_scan_bwd_args* a)
{
    return check_sizes(a) == GDR2_OK ? gdr2::scan_backward_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_scan_backward(const gdr2_scan_bwd_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    return hip_result(gdr2::launch_scan_backward(*a, (hipStream_t)stream), (hipStream_t)stream, "scan backward");
}

gdr2_status gdr2_norm_forward(const gdr2_norm_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->R == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_norm_forward(*a, (hipStream_t)stream), (hipStream_t)stream, "norm");
}

size_t gdr2_norm_backward_workspace_size(const gdr2_norm_bwd_args* a)
{
    return check_sizes(a) == GDR2_OK ? gdr2::norm_backward_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_norm_backward(const gdr2_norm_bwd_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    return hip_result(gdr2::launch_norm_backward(*a, (hipStream_t)stream), (hipStream_t)stream, "norm backward");
}

}  // extern "C"
