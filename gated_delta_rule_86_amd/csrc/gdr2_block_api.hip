// gdr2_block_api.hip -- the C ABI of the block operators (rows in 8 bits, norm
// with the residual's addition, gated linear recurrence): host-side validation
// and dispatch.  Every check runs before any launch; a failed check launches
// nothing and leaves the outputs untouched.
#include "gdr2_block.h"
#include "gdr2_checks.h"

namespace {

using namespace gdr2;

// The two buffers of rows in 8 bits.  `needed`: both have to be there.
void rows8_bufs(const gdr2_rows8& r, const char* codes, const char* scales, int64_t R, int64_t C, bool out, bool needed, Buf* b)
{
    b[0] = dense(codes, r.codes, mul(R, C), 1, out, needed || r.scales);
    b[1] = dense(scales, r.scales, mul(R, scale_count(C)), 1, out, needed || r.codes);
}

gdr2_status check_rows(int64_t R, int64_t C)
{
    if (R < 0)
        return set_error(GDR2_ERR_INVALID_ARG, "R must be >= 0");
    if (C <= 0)
        return set_error(GDR2_ERR_INVALID_ARG, "C must be positive (got %lld)", (long long)C);
    return R >= ((int64_t)1 << 40) ? set_error(GDR2_ERR_UNSUPPORTED, "2^40 or more rows") : GDR2_OK;
}

// ---- rows in 8 bits --------------------------------------------------------

gdr2_status validate(const gdr2_pack_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_rows(a->R, a->C));
    GDR2_TRY(check_dtype(a->dtype, a->reserved));
    GDR2_TRY(check_stride("x_stride", a->x_stride, a->C));
    Buf b[3];
    b[0] = rows_in("x", a->x, a->R, a->C, a->x_stride, elt(a->dtype));
    rows8_bufs(a->out, "codes", "scales", a->R, a->C, true, true, b + 1);
    return check_bufs(b, 3);
}

gdr2_status validate(const gdr2_unpack_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_rows(a->R, a->C));
    GDR2_TRY(check_dtype(a->dtype, a->reserved));
    GDR2_TRY(check_stride("C", a->C, a->C));
    Buf b[3];
    b[0] = dense("y", a->y, mul(a->R, a->C), elt(a->dtype), true);
    rows8_bufs(a->rows, "codes", "scales", a->R, a->C, false, true, b + 1);
    return check_bufs(b, 3);
}

// ---- norm with the residual's addition -------------------------------------

gdr2_status check_add_norm(int64_t R, int64_t C, int32_t dtype, int32_t res_dtype, int32_t kind, float eps)
{
    GDR2_TRY(check_rows(R, C));
    GDR2_TRY(check_dtype(dtype, 0));
    if (res_dtype != GDR2_F32 && res_dtype != GDR2_BF16)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown res_dtype %d", res_dtype);
    if (kind != GDR2_NORM_LAYER && kind != GDR2_NORM_RMS)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown kind %d", kind);
    if (!(eps >= 0.f) || std::isinf(eps))
        return set_error(GDR2_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (res_dtype != dtype && res_dtype != GDR2_F32)
        return set_error(GDR2_ERR_UNSUPPORTED, "the residual stream has the rows' dtype or is fp32");
    if (C > kAddNormMaxWidth)
        return set_error(GDR2_ERR_UNSUPPORTED, "rows may have at most %lld elements (got %lld)", (long long)kAddNormMaxWidth,
                         (long long)C);
    return GDR2_OK;
}

gdr2_status validate(const gdr2_add_norm_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_add_norm(a->R, a->C, a->dtype, a->res_dtype, a->kind, a->eps));
    GDR2_TRY(check_stride("x_stride", a->x_stride, a->C));
    if (a->residual)
        GDR2_TRY(check_stride("res_stride", a->res_stride, a->C));
    else if (a->R > 0 && a->res_dtype != a->dtype)
        return set_error(GDR2_ERR_INVALID_ARG, "res_dtype must be dtype without a residual");
    if (a->R > 0 && !a->h && !a->y && !a->y8.codes && !a->y8.scales && !a->h8.codes && !a->h8.scales)
        return set_error(GDR2_ERR_INVALID_ARG, "no output is given: h, y, y8 and h8 are NULL");
    const int64_t e = elt(a->dtype), er = elt(a->res_dtype), n = mul(a->R, a->C);
    Buf b[10] = {
        rows_in("x", a->x, a->R, a->C, a->x_stride, e),
        rows_in("residual", a->residual, a->R, a->C, a->res_stride, er, false),
        dense("weight", a->weight, a->C, 4, false, false),
        dense("bias", a->bias, a->C, 4, false, false),
        dense("h", a->h, n, er, true, false),
        dense("y", a->y, n, e, true, false),
    };
    rows8_bufs(a->y8, "y8.codes", "y8.scales", a->R, a->C, true, false, b + 6);
    rows8_bufs(a->h8, "h8.codes", "h8.scales", a->R, a->C, true, false, b + 8);
    return check_bufs(b, 10, a->res_stride == a->C ? "h" : "", a->res_stride == a->C ? "residual" : "");
}

gdr2_status check_sizes(const gdr2_add_norm_bwd_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    return check_add_norm(a->R, a->C, a->dtype, a->res_dtype, a->kind, a->eps);
}

gdr2_status validate(const gdr2_add_norm_bwd_args* a)
{
    GDR2_TRY(check_sizes(a));
    if (a->h && (a->h8.codes || a->h8.scales))
        return set_error(GDR2_ERR_INVALID_ARG, "h and h8 are both given");
    if (a->R > 0 && !a->dresidual && !a->dx)
        return set_error(GDR2_ERR_INVALID_ARG, "no output is given: dresidual and dx are NULL");
    const size_t need = add_norm_backward_workspace_bytes(*a);
    GDR2_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const int64_t e = elt(a->dtype), er = elt(a->res_dtype), n = mul(a->R, a->C);
    const bool packed = a->h8.codes || a->h8.scales;
    Buf b[11] = {
        dense("weight", a->weight, a->C, 4, false, false),
        dense("h", a->h, n, er, false, !packed),
        dense("dy", a->dy, n, e, false),
        dense("dh", a->dh, n, er, false, false),
        dense("dresidual", a->dresidual, n, er, true, false),
        dense("dx", a->dx, n, e, true, false),
        dense("dweight", a->dweight, a->C, 4, true, false),
        dense("dbias", a->dbias, a->C, 4, true, false),
        dense("workspace", a->workspace, (int64_t)need, 1, true),
    };
    rows8_bufs(a->h8, "h8.codes", "h8.scales", a->R, a->C, false, packed, b + 9);
    return check_bufs(b, 11, "dresidual", "dh");
}

// ---- gated linear recurrence -----------------------------------------------

// `rows`: x, r and i are there, with their strides.
gdr2_status check_glr(const gdr2_glr_args& a, bool backward, bool rows)
{
    if (a.B < 0 || a.T < 0)
        return set_error(GDR2_ERR_INVALID_ARG, "B, T must be >= 0");
    if (a.C <= 0)
        return set_error(GDR2_ERR_INVALID_ARG, "C must be positive (got %lld)", (long long)a.C);
    GDR2_TRY(check_dtype(a.dtype, 0));
    if (a.algo != GDR2_ALGO_AUTO && a.algo != GDR2_ALGO_STAGED && a.algo != GDR2_ALGO_SEGMENTED)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown algo %d", a.algo);
    if (a.C > kGlrMaxStride)
        return set_error(GDR2_ERR_UNSUPPORTED, "rows may have at most 2^22 elements (got %lld)", (long long)a.C);
    const struct {
        const char* name;
        int64_t ld;
    } strides[] = {{"x_stride", a.x_stride}, {"r_stride", a.r_stride}, {"i_stride", a.i_stride}};
    for (const auto& s : strides) {
        if (!rows)
            break;
        if (s.ld < a.C)
            return set_error(GDR2_ERR_INVALID_ARG, "%s must be at least the row's %lld elements (got %lld)", s.name, (long long)a.C,
                             (long long)s.ld);
        if (s.ld > kGlrMaxStride)
            return set_error(GDR2_ERR_UNSUPPORTED, "%s: rows may be at most 2^22 elements apart", s.name);
    }
    const int64_t n = a.offsets ? a.T : mul(a.B, a.T);
    if (a.B > ((int64_t)1 << 31) || a.T > ((int64_t)1 << 40) || n > ((int64_t)1 << 40) || glr_launch_groups(a, backward) >= kMaxGroups)
        return too_many();
    return GDR2_OK;
}

int64_t glr_rows(const gdr2_glr_args& a) { return a.B == 0 ? 0 : a.offsets ? a.T : a.B * a.T; }

// x, r, i, A and offsets
void glr_inputs(const gdr2_glr_args& a, bool rows, Buf* b)
{
    const int64_t e = elt(a.dtype), n = glr_rows(a);
    b[0] = rows_in("x", a.x, n, a.C, a.x_stride, e, rows);
    b[1] = rows_in("r", a.r, n, a.C, a.r_stride, e, rows);
    b[2] = rows_in("i", a.i, n, a.C, a.i_stride, e, rows);
    b[3] = dense("A", a.A, a.C, 4, false);
    b[4] = Buf{"offsets", a.offsets, mul(a.B + 1, 8), 8, false, false};
}

void glr_rows8(const gdr2_glr_args& a, bool out, bool needed, Buf* b)
{
    const int64_t n = glr_rows(a);
    const bool any = needed || a.x8.codes || a.x8.scales || a.r8.codes || a.r8.scales || a.i8.codes || a.i8.scales;
    rows8_bufs(a.x8, "x8.codes", "x8.scales", n, a.C, out, any, b);
    rows8_bufs(a.r8, "r8.codes", "r8.scales", n, a.C, out, any, b + 2);
    rows8_bufs(a.i8, "i8.codes", "i8.scales", n, a.C, out, any, b + 4);
}

int64_t glr_chunk_floats(const gdr2_glr_args& a) { return mul(gdr2_glr_chunk_count(a.B, a.T, a.offsets != nullptr), a.C); }

gdr2_status validate(const gdr2_glr_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    GDR2_TRY(check_glr(*a, false, true));
    const size_t need = glr_workspace_bytes(*a);
    GDR2_TRY(check_workspace(a->workspace, a->workspace_bytes, need));
    const int64_t st = mul(a->B, a->C);
    Buf b[16];
    glr_inputs(*a, true, b);
    b[5] = dense("h0", a->h0, st, 4, false, false);
    b[6] = dense("y", a->y, mul(glr_rows(*a), a->C), elt(a->dtype), true);
    b[7] = dense("h_out", a->h_out, st, 4, true, false);
    b[8] = dense("h_chunks", a->h_chunks, glr_chunk_floats(*a), 4, true, false);
    b[9] = dense("workspace", a->workspace, (int64_t)need, 1, true);
    glr_rows8(*a, true, false, b + 10);
    return check_bufs(b, 16, "h_out", "h0");
}

gdr2_status validate(const gdr2_glr_step_args* a)
{
    if (!a)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    if (a->N < 0)
        return set_error(GDR2_ERR_INVALID_ARG, "N must be >= 0");
    GDR2_TRY(check_rows(a->N, a->C));
    GDR2_TRY(check_dtype(a->dtype, a->reserved));
    GDR2_TRY(check_stride("x_stride", a->x_stride, a->C));
    GDR2_TRY(check_stride("r_stride", a->r_stride, a->C));
    GDR2_TRY(check_stride("i_stride", a->i_stride, a->C));
    const int64_t e = elt(a->dtype);
    const Buf b[] = {
        rows_in("x", a->x, a->N, a->C, a->x_stride, e),
        rows_in("r", a->r, a->N, a->C, a->r_stride, e),
        rows_in("i", a->i, a->N, a->C, a->i_stride, e),
        dense("A", a->A, a->C, 4, false),
        dense("state", a->state, mul(a->N, a->C), 4, true),
        dense("y", a->y, mul(a->N, a->C), e, true),
    };
    return check_bufs(b, 6);
}

// Rows in 8 bits stand in for x, r and i where none of these is given.
bool glr_packed(const gdr2_glr_args& a) { return !a.x && !a.r && !a.i; }

gdr2_status check_sizes(const gdr2_glr_bwd_args* p)
{
    if (!p)
        return set_error(GDR2_ERR_INVALID_ARG, "args is NULL");
    return check_glr(p->f, true, !glr_packed(p->f));
}

gdr2_status validate(const gdr2_glr_bwd_args* p)
{
    GDR2_TRY(check_sizes(p));
    const gdr2_glr_args& a = p->f;
    const bool packed = glr_packed(a) && (a.x8.codes || a.x8.scales || a.r8.codes || a.r8.scales || a.i8.codes || a.i8.scales);
    if (!glr_packed(a) && (a.x8.codes || a.r8.codes || a.i8.codes))
        return set_error(GDR2_ERR_INVALID_ARG, "x, r, i and x8, r8, i8 are both given");
    const size_t need = glr_backward_workspace_bytes(*p);
    GDR2_TRY(check_workspace(p->workspace, p->workspace_bytes, need));
    const int64_t e = elt(a.dtype), n = mul(glr_rows(a), a.C), st = mul(a.B, a.C);
    Buf b[20];
    glr_inputs(a, !packed, b);
    glr_rows8(a, false, packed, b + 5);
    b[11] = dense("h_chunks", a.h_chunks, glr_chunk_floats(a), 4, false);
    b[12] = dense("dy", p->dy, n, e, false);
    b[13] = dense("dh_out", p->dh_out, st, 4, false, false);
    b[14] = dense("dx", p->dx, n, e, true);
    b[15] = dense("dr", p->dr, n, e, true);
    b[16] = dense("di", p->di, n, e, true);
    b[17] = dense("dA", p->dA, a.C, 4, true);
    b[18] = dense("dh0", p->dh0, st, 4, true, false);
    b[19] = dense("workspace", p->workspace, (int64_t)need, 1, true);
    return check_bufs(b, 20, "dh0", "dh_out");
}

}  // namespace

extern "C" {

gdr2_status gdr2_pack_rows(const gdr2_pack_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->R == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_pack(*a, (hipStream_t)stream), (hipStream_t)stream, "pack");
}

gdr2_status gdr2_unpack_rows(const gdr2_unpack_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->R == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_unpack(*a, (hipStream_t)stream), (hipStream_t)stream, "unpack");
}

gdr2_status gdr2_add_norm_forward(const gdr2_add_norm_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->R == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_add_norm_forward(*a, (hipStream_t)stream), (hipStream_t)stream, "add_norm");
}

size_t gdr2_add_norm_backward_workspace_size(const gdr2_add_norm_bwd_args* a)
{
    return check_sizes(a) == GDR2_OK ? gdr2::add_norm_backward_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_add_norm_backward(const gdr2_add_norm_bwd_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    return hip_result(gdr2::launch_add_norm_backward(*a, (hipStream_t)stream), (hipStream_t)stream, "add_norm backward");
}

int64_t gdr2_glr_chunk_count(int64_t B, int64_t T, int packed)
{
    if (B <= 0 || T < 0)
        return 0;
    return packed ? T / GDR2_GLR_CHUNK + B : mul(B, T / GDR2_GLR_CHUNK + (T % GDR2_GLR_CHUNK != 0));
}

size_t gdr2_glr_workspace_size(const gdr2_glr_args* a)
{
    return a && check_glr(*a, false, true) == GDR2_OK ? gdr2::glr_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_glr_forward(const gdr2_glr_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->B == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_glr_forward(*a, (hipStream_t)stream), (hipStream_t)stream, "gated linear recurrence");
}

gdr2_status gdr2_glr_step(const gdr2_glr_step_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    if (a->N == 0)
        return GDR2_OK;
    return hip_result(gdr2::launch_glr_step(*a, (hipStream_t)stream), (hipStream_t)stream, "gated linear recurrence step");
}

size_t gdr2_glr_backward_workspace_size(const gdr2_glr_bwd_args* a)
{
    return check_sizes(a) == GDR2_OK ? gdr2::glr_backward_workspace_bytes(*a) : 0;
}

gdr2_status gdr2_glr_backward(const gdr2_glr_bwd_args* a, void* stream)
{
    GDR2_TRY(validate(a));
    return hip_result(gdr2::launch_glr_backward(*a, (hipStream_t)stream), (hipStream_t)stream, "gated linear recurrence backward");
}

}  // extern "C"
