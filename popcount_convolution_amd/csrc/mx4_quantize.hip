// Rows to microscaled 4-bit floats.
//
// A lane takes 8 values (16 or 32 bytes), the four lanes of a block of 32 share
// their largest magnitude by two swaps, its exponent is the scale, and the
// conversion instruction rounds a pair of values under it: about 20 vector
// instructions for 8 values of 16 bits, next to their 16 bytes.
//
// Bound by its bytes: 8193 x 8192 bf16 with the values, 304 MB, 46 us (6.6 TB/s; 51
// with loads that fill the caches), without them, 170 MB, 28 to 34 us.
// 32 x 4096: 3.6 us, a launch and one chain of a load and a store.
#include <hip/hip_runtime.h>

#include "host.h"
#include "mx4.h"

namespace bconv {

constexpr int kQuantThreads = 256;
static_assert(kQuantThreads == kListThreads);
constexpr int kQuantEach = 4;  // groups of 8 values a thread, requested together

struct QuantArgs {
    const void *x;
    uint8_t *codes, *scales;
    void *values;
    long long ldx;
    long long srow, sstep;  // bytes between the scales of rows and of steps
    uint32_t units;    // groups of 8 values of all rows, padding included
    uint32_t per_row;  // of one row
    int cols;
    uint32_t groups;  // workgroups that quantise; one more makes the list
    RowBlocks list;
};

// max over the 4 lanes of a block
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true);  // quad_perm [1,0,3,2]
    v = o > v ? o : v;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true);           // quad_perm [2,3,0,1]
    return o > v ? o : v;
}

// What 8 codes under a scale byte stand for, in `DT`.
template <int DT> __device__ __forceinline__ Eight<DT> from_codes(uint32_t c, uint32_t byte)
{
    const float s = __builtin_bit_cast(float, byte << 23);
    Eight<DT> e;
    if constexpr (DT == BCONV_F32) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3)};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e.q[i >> 2][i & 3] = byte == 255 ? 0x7fc00000u : __builtin_bit_cast(uint32_t, (float)v[i >> 1][i & 1]);
    } else if constexpr (DT == BCONV_F16) {
        const f16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3)};
#pragma unroll
        for (int i = 0; i < 4; ++i) e.q[0][i] = byte == 255 ? 0x7e007e00u : __builtin_bit_cast(uint32_t, v[i]);
    } else {
        const bf16x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1),
                             __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3)};
#pragma unroll
        for (int i = 0; i < 4; ++i) e.q[0][i] = byte == 255 ? 0x7fc07fc0u : __builtin_bit_cast(uint32_t, v[i]);
    }
    return e;
}

template <int DT> __device__ __forceinline__ void store_values(typename Elem<DT>::type *p, const Eight<DT> &e, int left)
{
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < (DT == BCONV_F32 ? 2 : 1); ++i) reinterpret_cast<u32x4_any *>(p)[i] = e.q[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i >= left) break;
        if constexpr (DT == BCONV_F32) p[i] = __builtin_bit_cast(float, (uint32_t)e.q[i >> 2][i & 3]);
        else reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(e.q[0][i >> 1] >> (16 * (i & 1)));
    }
}

template <int DT, bool VALUES> __global__ __launch_bounds__(kQuantThreads) void mx4_quantize_kernel(QuantArgs a)
{
    typedef typename Elem<DT>::type T;
    if (blockIdx.x == a.groups) {
        make_row_blocks(a.list);
        return;
    }
    Eight<DT> v[kQuantEach];
    uint32_t row[kQuantEach], at[kQuantEach];
#pragma unroll
    for (int j = 0; j < kQuantEach; ++j) {
        const uint32_t unit = (blockIdx.x * kQuantEach + j) * kQuantThreads + threadIdx.x;
        row[j] = unit / a.per_row;
        at[j] = (unit - row[j] * a.per_row) * 8;
        const int left = unit < a.units ? a.cols - (int)at[j] : 0;
        v[j] = load_values<DT, true>(static_cast<const T *>(a.x) + (left > 0 ? (long long)row[j] * a.ldx + at[j] : 0), left);
    }
#pragma unroll
    for (int j = 0; j < kQuantEach; ++j) {
        const uint32_t unit = (blockIdx.x * kQuantEach + j) * kQuantThreads + threadIdx.x;
        const uint32_t byte = scale_byte<DT>(block_max(largest<DT>(v[j])));
        const uint32_t c = to_codes<DT>(v[j], byte);
        if (unit >= a.units) continue;  // whole blocks: units are a multiple of 4
        reinterpret_cast<uint32_t *>(a.codes)[unit] = c;
        if ((threadIdx.x & 3) == 0) a.scales[row[j] * a.srow + (at[j] / kStep) * a.sstep + at[j] / 32 % 8] = (uint8_t)byte;
        if constexpr (VALUES) {
            const int left = a.cols - (int)at[j];
            if (left > 0)
                store_values<DT>(static_cast<T *>(a.values) + (long long)row[j] * a.cols + at[j], from_codes<DT>(c, byte), left);
        }
    }
}

template <int DT> static void launch_quantize(const QuantArgs &a, hipStream_t s)
{
    const unsigned grid = a.groups + (a.list.list ? 1 : 0);
    if (a.values) hipLaunchKernelGGL((mx4_quantize_kernel<DT, true>), dim3(grid), dim3(kQuantThreads), 0, s, a);
    else hipLaunchKernelGGL((mx4_quantize_kernel<DT, false>), dim3(grid), dim3(kQuantThreads), 0, s, a);
}

hipError_t mx4_quantize_rows(hipStream_t s, long long rows, int cols, int dtype, const void *x, long long ldx,
                             uint8_t *codes, uint8_t *scales, long long srow, long long sstep, void *values,
                             const RowBlocks &blocks)
{
    const int es = dtype == BCONV_F32 ? 4 : 2;
    const long long per_row = mx4_padded(cols) / 8;
    const long long slab = (1LL << 30) / per_row;  // rows a launch: units in 32 bits
    for (long long first = 0; first < rows; first += slab) {
        const long long n = rows - first < slab ? rows - first : slab;
        QuantArgs a{};
        a.x = static_cast<const char *>(x) + first * ldx * es;
        a.codes = codes + first * per_row * 4;
        a.scales = scales + first * srow;
        a.values = values ? static_cast<char *>(values) + first * cols * es : nullptr;
        a.ldx = ldx;
        a.srow = srow;
        a.sstep = sstep;
        a.units = (uint32_t)(n * per_row);
        a.per_row = (uint32_t)per_row;
        a.cols = cols;
        a.groups = (a.units + kQuantThreads * kQuantEach - 1) / (kQuantThreads * kQuantEach);
        if (first == 0) a.list = blocks;
        switch (dtype) {
        case BCONV_F32: launch_quantize<BCONV_F32>(a, s); break;
        case BCONV_F16: launch_quantize<BCONV_F16>(a, s); break;
        default: launch_quantize<BCONV_BF16>(a, s); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace bconv

using bconv::fail;
using bconv::ranges_overlap;

extern "C" bconv_status_t bconv_mx4_quantize(void *stream, int32_t rows, int32_t cols, int32_t dtype, const void *x,
                                             int64_t ldx, uint8_t *codes, uint8_t *scales, void *values)
{
    const int es = dtype == BCONV_F32 ? 4 : dtype == BCONV_F16 || dtype == BCONV_BF16 ? 2 : 0;
    if (!es) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
    if (rows < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows must be >= 0");
    if (cols < 1 || cols > (1 << 20)) return fail(BCONV_ERR_INVALID_ARGUMENT, "cols must be in [1, %d]", 1 << 20);
    if (ldx < cols || ldx > bconv::kMaxStride) return fail(BCONV_ERR_INVALID_ARGUMENT, "ldx must be in [cols, 2^30]");
    if (rows == 0) return BCONV_OK;
    if (!x || !codes || !scales) return fail(BCONV_ERR_INVALID_ARGUMENT, "x, codes and scales must not be NULL");
    if (((uintptr_t)x | (uintptr_t)values) % es) return fail(BCONV_ERR_INVALID_ARGUMENT, "x/values not aligned to an element");
    if ((uintptr_t)codes % 16 || (uintptr_t)scales % 8)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned, scales 8-byte");
    const long long padded = bconv::mx4_padded(cols);
    const struct { const void *p; size_t n; } spans[] = {
        {x, ((size_t)(rows - 1) * ldx + cols) * es}, {codes, (size_t)rows * (padded / 2)}, {scales, (size_t)rows * (padded / 32)},
        {values, values ? (size_t)rows * cols * es : 0}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (spans[i].n && ranges_overlap(spans[i].p, spans[i].n, spans[j].p, spans[j].n))
                return fail(BCONV_ERR_INVALID_ARGUMENT, "codes, scales and values must overlap neither x nor each other");
    const hipError_t e = bconv::mx4_quantize_rows(static_cast<hipStream_t>(stream), rows, cols, dtype, x, ldx, codes, scales, padded / 32, 8, values, bconv::RowBlocks{});
    if (e != hipSuccess) return bconv::hip_fail(e, "mx4 quantisation kernel");
    return BCONV_OK;
}
