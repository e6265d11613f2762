// gdr2_rows8.hip -- rows into 8 bits (e4m3 codes, one power of two per 32
// columns) and back.
//
//   e = min { e >= -127 : max_block |v| <= 448 2^e },  code = e4m3(v 2^-e)
//
// Memory bounds both: 3 bytes an element of bf16 rows.  A lane holds 8 columns
// (one access of 16 bytes), four lanes a block.  32768 rows of 2048 bf16 in 42 us
// and 32 us back, 4.9 and 6.3 TB/s (a large copy 5.15); a slice of 10007 rows of
// 1003 fp32, whose vectors begin at any element, in 10 and 11 us.
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
__device__ __forceinline__ int left_of(int64_t C, int64_t c) { return C - c >= 8 ? 8 : (int)(C - c); }

template <typename T> __global__ __launch_bounds__(256) void pack_kernel(gdr2_pack_args a, int64_t items)
{
    const int64_t nb = scale_count(a.C), step = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < items; at += step) {
        const Place p = place_of(at, nb * 4, a.R == 1);
        const int64_t c = p.item * 8;
        const int n = left_of(a.C, c);
        Row8<T> raw;
        raw.load((const T*)a.x + p.row * a.x_stride + c, n);
        float v[8];
        raw.get(v);
        const int amax = block_max<8>(v, n), e = block_exponent(amax);
        Codes8 k;
        k.pack(v, amax, e);
        k.store((uint8_t*)a.out.codes + p.row * a.C + c, n);
        if (p.item % 4 == 0)
            ((uint8_t*)a.out.scales)[p.row * nb + p.item / 4] = (uint8_t)(e + 127);
    }
}

template <typename T> __global__ __launch_bounds__(256) void unpack_kernel(gdr2_unpack_args a, int64_t items)
{
    const int64_t nb = scale_count(a.C), per = (a.C + 7) / 8, step = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < items; at += step) {
        const Place p = place_of(at, per, a.R == 1);
        const int64_t c = p.item * 8;
        const int n = left_of(a.C, c);
        Codes8 k;
        k.load((const uint8_t*)a.rows.codes + p.row * a.C + c, n);
        float v[8];
        k.get(((const uint8_t*)a.rows.scales)[p.row * nb + c / kRows8], v);
        Row8<T>::store((T*)a.y + p.row * a.C + c, v, n);
    }
}

// Eight workgroups per compute unit, then the items are walked.
unsigned grid_of(int64_t items) { return (unsigned)std::min(ceil_div(items, 256), (int64_t)device_cu_count() * 8); }

}  // namespace

hipError_t launch_pack(const gdr2_pack_args& args, hipStream_t stream)
{
    gdr2_pack_args a = args;
    if (a.x_stride == a.C && a.C % kRows8 == 0) {
        a.C *= a.R;
        a.R = 1;
    }
    const int64_t items = a.R * scale_count(a.C) * 4;
    if (a.dtype == GDR2_BF16)
        hipLaunchKernelGGL((pack_kernel<bf16>), dim3(grid_of(items)), dim3(256), 0, stream, a, items);
    else
        hipLaunchKernelGGL((pack_kernel<float>), dim3(grid_of(items)), dim3(256), 0, stream, a, items);
    return hipGetLastError();
}

hipError_t launch_unpack(const gdr2_unpack_args& args, hipStream_t stream)
{
    gdr2_unpack_args a = args;
    if (a.C % kRows8 == 0) {
        a.C *= a.R;
        a.R = 1;
    }
    const int64_t items = a.R * ceil_div(a.C, 8);
    if (a.dtype == GDR2_BF16)
        hipLaunchKernelGGL((unpack_kernel<bf16>), dim3(grid_of(items)), dim3(256), 0, stream, a, items);
    else
        hipLaunchKernelGGL((unpack_kernel<float>), dim3(grid_of(items)), dim3(256), 0, stream, a, items);
    return hipGetLastError();
}

}  // namespace gdr2
