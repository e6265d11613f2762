// gdr2_rows8.hip -- rows into 8 bits (e4m3 codes, one power of two per 32
// columns) and back.
//
//   e = min { e >= -127 : max_block |v| <= 448 2^e },  code = e4m3(v 2^-e)
//
// Memory bounds both: 3 bytes an element of bf16 rows, and two operations on
// the matrix of a block's lanes.  A lane holds 8 columns, four lanes a block
// (one column and 32 lanes where rows are not whole, aligned vectors).
#include <algorithm>

#include "gdr2_block.h"

namespace gdr2 {

namespace {

// Item `at` of rows of `per` items each.  Dense rows of whole blocks are one
// long row, which needs no division.
struct Place {
    int64_t row, item;
};
__device__ __forceinline__ Place place_of(int64_t at, int64_t per, bool one_row)
{
    if (one_row)
        return {0, at};
    const int64_t row = (at | per) >> 32 ? at / per : (int64_t)((uint32_t)at / (uint32_t)per);
    return {row, at - row * per};
}

template <typename T, int V> __global__ __launch_bounds__(256) void pack_kernel(gdr2_pack_args a, int64_t items)
{
    constexpr int LPB = kRows8 / V;
    const int64_t nb = scale_count(a.C), per = nb * LPB, step = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < items; at += step) {
        const Place p = place_of(at, per, a.R == 1);
        const int64_t c = p.item * V;
        const bool in = c < a.C;
        RowPart<T, V> raw;
        if (in)
            raw.load((const T*)a.x + p.row * a.x_stride + c);
        else
            raw.zero();
        float v[V];
        raw.get(v);
        const int amax = block_max<V>(v, in), e = block_exponent(amax);
        Codes<V> k;
        k.pack(v, amax, e);
        if (in)
            k.store((uint8_t*)a.out.codes + p.row * a.C + c);
        if (p.item % LPB == 0)
            ((uint8_t*)a.out.scales)[p.row * nb + p.item / LPB] = (uint8_t)(e + 127);
    }
}

template <typename T, int V> __global__ __launch_bounds__(256) void unpack_kernel(gdr2_unpack_args a, int64_t items)
{
    const int64_t nb = scale_count(a.C), per = (a.C + V - 1) / V, step = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < items; at += step) {
        const Place p = place_of(at, per, a.R == 1);
        const int64_t c = p.item * V;
        Codes<V> k;
        k.load((const uint8_t*)a.rows.codes + p.row * a.C + c);
        float v[V];
        k.get(((const uint8_t*)a.rows.scales)[p.row * nb + c / kRows8], v);
        RowPart<T, V>::store((T*)a.y + p.row * a.C + c, v);
    }
}

// Eight workgroups per compute unit, then the items are walked.
unsigned grid_of(int64_t items) { return (unsigned)std::min(ceil_div(items, 256), (int64_t)device_cu_count() * 8); }

template <typename T, int V> hipError_t pack_v(gdr2_pack_args a, hipStream_t stream)
{
    if (a.x_stride == a.C && a.C % kRows8 == 0) {
        a.C *= a.R;
        a.R = 1;
    }
    const int64_t items = a.R * scale_count(a.C) * (kRows8 / V);
    hipLaunchKernelGGL((pack_kernel<T, V>), dim3(grid_of(items)), dim3(256), 0, stream, a, items);
    return hipGetLastError();
}

template <typename T, int V> hipError_t unpack_v(gdr2_unpack_args a, hipStream_t stream)
{
    if (a.C % kRows8 == 0) {
        a.C *= a.R;
        a.R = 1;
    }
    const int64_t items = a.R * ceil_div(a.C, V);
    hipLaunchKernelGGL((unpack_kernel<T, V>), dim3(grid_of(items)), dim3(256), 0, stream, a, items);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pack(const gdr2_pack_args& a, hipStream_t stream)
{
    const bool bf = a.dtype == GDR2_BF16, wide = rows_in_eights(a.x, a.x_stride, a.C, a.dtype);
    if (bf)
        return wide ? pack_v<bf16, 8>(a, stream) : pack_v<bf16, 1>(a, stream);
    return wide ? pack_v<float, 8>(a, stream) : pack_v<float, 1>(a, stream);
}

hipError_t launch_unpack(const gdr2_unpack_args& a, hipStream_t stream)
{
    const bool wide = a.C % 8 == 0;
    if (a.dtype == GDR2_BF16)
        return wide ? unpack_v<bf16, 8>(a, stream) : unpack_v<bf16, 1>(a, stream);
    return wide ? unpack_v<float, 8>(a, stream) : unpack_v<float, 1>(a, stream);
}

}  // namespace gdr2
