// gdr2_checks.h -- the argument checks that the entry points beside the
// recurrence share (host only): buffers, strides, workspaces.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "gdr2.h"
#include "gdr2_internal.h"

namespace gdr2 {

// GDR2_OK, or GDR2_ERR_HIP with the error's text; GDR2_DEBUG=1 waits for the
// work first, as for the recurrence's entry points.
inline gdr2_status hip_result(hipError_t e, hipStream_t stream, const char* what)
{
    static const bool wait = [] {
        const char* v = std::getenv("GDR2_DEBUG");
        return v && v[0] && v[0] != '0';
    }();
    if (e == hipSuccess && wait)
        e = hipStreamSynchronize(stream);
    return e == hipSuccess ? GDR2_OK : set_error(GDR2_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int64_t kHuge = (int64_t)1 << 62;
// Elements of a row, and between two rows.  The scan's prompt and gradient kernels form offsets
// within 32 rows in 32 bits of bytes; the others in 64 bits.
constexpr int64_t kMaxWidth = (int64_t)1 << 24, kMaxStride = (int64_t)1 << 40, kScanMaxStride = (int64_t)1 << 24;

// One buffer of a call: its bytes from the first to the last element.
struct Buf {
    const char* name;
    const void* p;
    int64_t bytes;   // 0: nothing to read or write, the pointer may be NULL
    int align;
    bool needed;
    bool out;
};

// Saturating product of non-negative sizes.
inline int64_t mul(int64_t a, int64_t b)
{
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) || r > kHuge ? kHuge : r;
}

inline int64_t elt(int32_t dtype) { return dtype == GDR2_BF16 ? 2 : 4; }

// rows of `width` elements, `stride` apart
inline Buf rows_in(const char* name, const void* p, int64_t rows, int64_t width, int64_t stride, int64_t e, bool needed = true)
{
    const int64_t n = rows > 0 ? mul(rows - 1, stride) : 0;
    return {name, p, rows > 0 ? (n >= kHuge ? kHuge : mul(n + width, e)) : 0, (int)e, needed, false};
}
inline Buf dense(const char* name, const void* p, int64_t n, int64_t e, bool out, bool needed = true)
{
    return {name, p, mul(n, e), 16, needed, out};
}

// NULL, alignment, size and overlap of every buffer.  Outputs overlap
// nothing, except the pair (alias_a, alias_b), which may be the same pointer.
inline gdr2_status check_bufs(const Buf* b, int n, const char* alias_a = "", const char* alias_b = "")
{
    for (int i = 0; i < n; ++i) {
        if (!b[i].p) {
            if (b[i].needed && b[i].bytes > 0)
                return set_error(GDR2_ERR_INVALID_ARG, "%s is NULL", b[i].name);
            continue;
        }
        if (b[i].bytes >= kHuge)
            return set_error(GDR2_ERR_INVALID_ARG, "%s: size overflows", b[i].name);
        if (reinterpret_cast<uintptr_t>(b[i].p) % (unsigned)b[i].align)
            return set_error(GDR2_ERR_INVALID_ARG, "%s is not %d-byte aligned", b[i].name, b[i].align);
    }
    auto same = [](const char* x, const char* y) {
        while (*x && *x == *y)
            ++x, ++y;
        return *x == *y;
    };
    for (int i = 0; i < n; ++i) {
        if (!b[i].out || !b[i].p || b[i].bytes == 0)
            continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || !b[j].p || b[j].bytes == 0 || (b[j].out && j < i))
                continue;
            const uintptr_t x = reinterpret_cast<uintptr_t>(b[i].p), y = reinterpret_cast<uintptr_t>(b[j].p);
            if (x == y && same(b[i].name, alias_a) && same(b[j].name, alias_b))
                continue;
            if (x < y + (uintptr_t)b[j].bytes && y < x + (uintptr_t)b[i].bytes)
                return set_error(GDR2_ERR_INVALID_ARG, "%s overlaps %s", b[i].name, b[j].name);
        }
    }
    return GDR2_OK;
}

inline gdr2_status check_dtype(int32_t dtype, int32_t reserved)
{
    if (dtype != GDR2_F32 && dtype != GDR2_BF16)
        return set_error(GDR2_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (reserved != 0)
        return set_error(GDR2_ERR_INVALID_ARG, "reserved field must be 0");
    return GDR2_OK;
}

inline gdr2_status check_stride(const char* name, int64_t stride, int64_t width, int64_t most = kMaxStride)
{
    if (stride < width)
        return set_error(GDR2_ERR_INVALID_ARG, "%s must be at least the row's %lld elements (got %lld)", name,
                         (long long)width, (long long)stride);
    if (width > kMaxWidth)
        return set_error(GDR2_ERR_UNSUPPORTED, "rows may have at most 2^24 elements (got %lld)", (long long)width);
    if (stride > most)
        return set_error(GDR2_ERR_UNSUPPORTED, "%s: rows may be at most 2^%d elements apart", name, most == kMaxStride ? 40 : 24);
    return GDR2_OK;
}

inline gdr2_status too_many() { return set_error(GDR2_ERR_UNSUPPORTED, "too many workgroups for one launch"); }

inline gdr2_status check_workspace(const void* p, size_t given, size_t need)
{
    if (need > 0 && (!p || given < need))
        return set_error(GDR2_ERR_WORKSPACE, "workspace of %zu bytes required, %zu given", need, p ? given : (size_t)0);
    return GDR2_OK;
}

#define GDR2_TRY(x)                    \
    do {                               \
        const gdr2_status s_ = (x);    \
        if (s_ != GDR2_OK)             \
            return s_;                 \
    } while (0)

}  // namespace gdr2
