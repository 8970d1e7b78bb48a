// Device helpers of the microscaled 4-bit operators: blocks of 32 values to
// codes and a power of two, and the layouts that the kernels share.  Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bconv_mx4.h"
#include "q4_device.h"

namespace bconv {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
// The same in memory at any element's address: global memory takes wide loads
// and stores at any alignment, in one instruction.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// Inputs of one step of the products: two 16 x 16 x 128 matrix instructions.
// Lane (row r = lane & 15, lg = lane >> 4) of a step holds the two blocks
// 64 lg .. 64 lg + 63 of its row, the first for the first instruction.  The sum
// over k may be taken in any order, as long as both operands agree; this one
// makes a lane's codes 32 and its scales 2 consecutive bytes of a quantised row.
constexpr int kStep = BCONV_MX4_PAD;

__host__ __device__ constexpr long long mx4_padded(long long cols)
{
    return (cols + BCONV_MX4_PAD - 1) / BCONV_MX4_PAD * BCONV_MX4_PAD;
}

// Elements between rows at most: the bytes of a call's rows stay below 2^63.
constexpr long long kMaxStride = 1LL << 30;

// (token, choice) pairs of a call at most, so rows of experts too.
constexpr long long kMaxPairs = 1LL << 27;

// 8 consecutive values of one row as loaded.
template <int DT> struct Eight {
    u32x4 q[DT == BCONV_F32 ? 2 : 1];
};

// Those of them that are in the row, zeros for the rest (`left` of them remain).
// ONCE: nothing here reads them again.
template <int DT, bool ONCE = false> __device__ __forceinline__ Eight<DT> load_values(const typename Elem<DT>::type *p, int left)
{
    Eight<DT> e;
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < (DT == BCONV_F32 ? 2 : 1); ++i) {
            const u32x4_any *q = reinterpret_cast<const u32x4_any *>(p) + i;
            if constexpr (ONCE) e.q[i] = __builtin_nontemporal_load(q);
            else e.q[i] = *q;
        }
        return e;
    }
    if constexpr (DT == BCONV_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e.q[i >> 2][i & 3] = i < left ? __builtin_bit_cast(uint32_t, p[i]) : 0u;
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            e.q[0][i] = (2 * i < left ? (uint32_t)h[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)h[2 * i + 1] << 16 : 0u);
    }
    return e;
}

// The largest magnitude of some values, as bits that order like it: of fp32, or
// of the 16-bit type.
template <int DT> __device__ __forceinline__ uint32_t largest(const Eight<DT> &e)
{
    if constexpr (DT == BCONV_F32) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = e.q[i >> 2][i & 3] & 0x7fffffffu;
            m = a > m ? a : m;
        }
        return m;
    } else {
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, (uint32_t)(e.q[0][i] & 0x7fff7fffu)));
        return m[0] > m[1] ? m[0] : m[1];
    }
}

// A block's scale byte from the bits of its largest magnitude: the exponent
// field of that as fp32, less 2, at least 0; 255 for infinities and NaN.
template <int DT> __device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    uint32_t bits = top;
    if constexpr (DT == BCONV_BF16) bits = top << 16;
    if constexpr (DT == BCONV_F16)
        bits = __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)top));
    const int field = (int)(bits >> 23);
    return field == 255 ? 255u : (uint32_t)(field > 2 ? field - 2 : 0);
}

// Codes of 8 values under a scale byte.  The conversion divides by the power of
// two of its scale operand's exponent field (0 is 2^-127), rounds to the nearest,
// ties to even, and saturates: compared with the definition for every exponent.
template <int DT> __device__ __forceinline__ uint32_t to_codes(const Eight<DT> &e, uint32_t byte)
{
    const float s = __builtin_bit_cast(float, byte << 23);
    uint32_t c = 0;
    if constexpr (DT == BCONV_F32) {
        const f32x4 a = __builtin_bit_cast(f32x4, e.q[0]), b = __builtin_bit_cast(f32x4, e.q[1]);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[0], b[1], s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[2], b[3], s, 3);
    } else if constexpr (DT == BCONV_F16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)e.q[0][0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)e.q[0][1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)e.q[0][2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)e.q[0][3]), s, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)e.q[0][0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)e.q[0][1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)e.q[0][2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)e.q[0][3]), s, 3);
    }
    return byte == 255 ? 0u : c;
}

// D += A B over 128 k of 16 x 16 results; `S` is the byte of the scale operands
// that belongs to these k.
template <int S> __device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c)
{
    const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    // cbsz = blgp = 4: e2m1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, S, (int)sa, S, (int)sb);
}

// D += A B over 64 k of 32 x 32 results, with byte `S` of the scale operands.
__device__ __forceinline__ f32x16 mfma_mx4_32(int S, u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 c)
{
    const i32x8 a8 = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 b8 = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    switch (S) {  // known where it is called
    case 0: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 0, (int)sa, 0, (int)sb);
    case 1: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 1, (int)sa, 1, (int)sb);
    case 2: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 2, (int)sa, 2, (int)sb);
    default: return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, 3, (int)sa, 3, (int)sb);
    }
}

// Result rows [begin, end) of expert f; f = experts: those of none.
struct Span {
    int begin, end;
};

__device__ __forceinline__ Span expert_rows(const int *offsets, int experts, int rows, int f)
{
    auto inside = [&](int o) { return o < 0 ? 0 : o > rows ? rows : o; };
    return {inside(offsets[f]), f < experts ? inside(offsets[f + 1]) : rows};
}

// The rows that a workgroup of a product takes, of expert f (experts: of none),
// and the blocks that are taken together: `group` / 32 is the first of them,
// `group` % 32 how many, all of the same expert.
struct RowBlock {
    int f, begin, end, group;
};

constexpr int kRowGroup = 16;  // at most

// Rows of all experts in blocks of up to `size`, expert by expert, those of none
// last: list[0].f is their number, they follow (at most row_blocks_most(); offsets
// that do not ascend could ask for more, which are left out).
struct RowBlocks {
    const int *offsets;
    RowBlock *list;  // or nullptr: none is wanted
    int experts, rows, size;
};

__host__ __device__ inline int row_blocks_most(int rows, int experts, int size)
{
    return (rows + size - 1) / size + experts + 1;
}

constexpr int kListThreads = 256;

// By one workgroup; a thread takes consecutive experts.
__device__ __forceinline__ void make_row_blocks(const RowBlocks &b)
{
    __shared__ int sums[kListThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int each = b.experts / kListThreads + 1, f0 = threadIdx.x * each;
    int count = 0;
    for (int f = f0; f < f0 + each && f <= b.experts; ++f) {
        const Span s = expert_rows(b.offsets, b.experts, b.rows, f);
        count += s.end > s.begin ? (s.end - s.begin + b.size - 1) / b.size : 0;
    }
    int upto = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(upto, d);
        if (lane >= d) upto += u;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - count;
    for (int w = 0; w < wave; ++w) at += sums[w];
    const int most = row_blocks_most(b.rows, b.experts, b.size);
    for (int f = f0; f < f0 + each && f <= b.experts; ++f) {
        const Span s = expert_rows(b.offsets, b.experts, b.rows, f);
        const int blocks = s.end > s.begin ? (s.end - s.begin + b.size - 1) / b.size : 0;
        const int held = blocks < most - at ? blocks : most - at;
        for (int i = 0; i < held; ++i) {
            const int r = s.begin + i * b.size, first = i / kRowGroup * kRowGroup;
            b.list[1 + at + i] = {f, r, s.end - r < b.size ? s.end : r + b.size,
                                  (at + first) * 32 + (held - first < kRowGroup ? held - first : kRowGroup)};
        }
        at += blocks;
    }
    if (threadIdx.x == kListThreads - 1) b.list[0].f = at < most ? at : most;
}

// Launches the quantisation of rows (see bconv_mx4_quantize); arguments are
// checked by the caller.  The 8 scales of a row's step are together, `srow`
// bytes from the next row's, `sstep` from the next step's.  One more workgroup makes `blocks`.
hipError_t mx4_quantize_rows(hipStream_t s, long long rows, int cols, int dtype, const void *x, long long ldx,
                             uint8_t *codes, uint8_t *scales, long long srow, long long sstep, void *values, const RowBlocks &blocks);

}  // namespace bconv
