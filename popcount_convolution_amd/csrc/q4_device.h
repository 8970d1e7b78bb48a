// Device helpers shared by the 4-bit operators: element types, matrix-core
// operands from packed 4-bit codes, exact splits of fp32 operands.  Not part
// of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bconv_q4.h"

namespace bconv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Element type of each bconv_dtype_t.
template <int DT> struct Elem;
template <> struct Elem<BCONV_F32> { typedef float type; };
template <> struct Elem<BCONV_F16> { typedef _Float16 type; };
template <> struct Elem<BCONV_BF16> { typedef __bf16 type; };

// 16-byte matrix-core operands a value takes: fp32 two fp16 parts (see Range),
// 16-bit types one, as they are.
template <int DT> constexpr int kSplit = DT == BCONV_F32 ? 2 : 1;

// One lane's operand of v_mfma_f32_16x16x32: 8 consecutive k of one row or
// column, for each part of the split.
template <int DT> struct Operand {
    u32x4 part[kSplit<DT>];
};

template <int DT> __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT != BCONV_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

template <int DT> __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (DT != BCONV_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// a . b + c over the parts of b (a is exact in one part), smallest part first.
template <int DT> __device__ __forceinline__ f32x4 mfma_parts(u32x4 a, const Operand<DT> &b, f32x4 c)
{
#pragma unroll
    for (int p = kSplit<DT> - 1; p >= 0; --p) c = mfma16<DT>(a, b.part[p], c);
    return c;
}

// The largest of four lanes' bits 16 apart (of non-negative floats as well).
__device__ __forceinline__ uint32_t lane_groups_max_bits(uint32_t v)
{
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = a[0] > a[1] ? a[0] : a[1];
    const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return b[0] > b[1] ? b[0] : b[1];
}

// The power of two `to` that brings values up to a largest magnitude below
// 2^(BITS + 1), for splitting them, and its inverse `from`.  Multiplying by either is
// exact.  Below 2^LEAST the largest magnitude is taken as that (so that both stay
// normal numbers).
//
// A value x times `to` is split into h = fp16(x), l = fp16(x - h): x - h is
// exact and at most 2^-11 x, a multiple of x's last bit, of which l holds all but
// the last in the upper half of that range.  So h + l is x to 2^-23 (23 of fp32's 24
// bits; three values in four are exact), as long as l is a normal number; below that
// its error is at most 2^-25, that is 2^-(25 + BITS) of the largest value.  Two products then stand for an
// fp32 product (exact bf16 parts would take three, and 8 instructions a value
// instead of 3).
template <int BITS, int LEAST = BITS - 126> struct Range {
    static_assert(LEAST >= BITS - 126 && BITS < 16);
    float to, from;
    __device__ __forceinline__ explicit Range(uint32_t top)
    {
        uint32_t e = top >> 23;
        e = e < 127 + LEAST ? 127 + LEAST : e;
        to = __uint_as_float((254 + BITS - e) << 23);
        from = __uint_as_float((e - BITS) << 23);
    }
};

// A pair of values times `to`, split as above.
__device__ __forceinline__ void split_pair(float x0, float x1, float to, uint32_t &h, uint32_t &l)
{
    const f16x2 r = {(_Float16)(x0 * to), (_Float16)(x1 * to)};
    h = __builtin_bit_cast(uint32_t, r);
    asm("" : "+v"(h));  // or the compiler converts each value once more
    const f16x2 q = __builtin_bit_cast(f16x2, h);
    const f16x2 d = {(_Float16)__builtin_fmaf(x0, to, -(float)q[0]), (_Float16)__builtin_fmaf(x1, to, -(float)q[1])};
    l = __builtin_bit_cast(uint32_t, d);
}

// 8 consecutive elements as loaded.
template <int DT> struct Raw {
    u32x4 v[DT == BCONV_F32 ? 2 : 1];
};

// 16-byte loads; p is 16-byte aligned.
template <int DT> __device__ __forceinline__ Raw<DT> load_raw(const typename Elem<DT>::type *p)
{
    Raw<DT> r;
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
    r.v[0] = q[0];
    if constexpr (DT == BCONV_F32) r.v[1] = q[1];
    return r;
}

// Element loads, for any alignment; elements at or past len (of a row that p is
// k into) are 0.
template <int DT>
__device__ __forceinline__ Raw<DT> load_raw_masked(const typename Elem<DT>::type *p, int k, int len)
{
    Raw<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == BCONV_F32 ? 2 : 1); ++i) r.v[i] = u32x4{0, 0, 0, 0};
    if (k >= len) return r;
    if constexpr (DT == BCONV_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i >> 2][i & 3] = k + i < len ? __float_as_uint(p[i]) : 0u;
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = k + 2 * i < len ? h[2 * i] : 0u, b = k + 2 * i + 1 < len ? h[2 * i + 1] : 0u;
            r.v[0][i] = a | (b << 16);
        }
    }
    return r;
}

// 8 consecutive elements at p (offset k of a row of length len); elements at or
// past len are 0.  `vec`: p is 16-byte aligned for k % 8 == 0.
template <int DT>
__device__ __forceinline__ Raw<DT> load_eight(const typename Elem<DT>::type *p, int k, int len, bool vec)
{
    return vec && k + 8 <= len ? load_raw<DT>(p) : load_raw_masked<DT>(p, k, len);
}

template <int DT> __device__ __forceinline__ Raw<DT> zero_raw()
{
    Raw<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == BCONV_F32 ? 2 : 1); ++i) r.v[i] = u32x4{0, 0, 0, 0};
    return r;
}

// N runs of 8 elements as operands.  fp32: times a power of two common to the
// four lanes that hold a row or column, and `from` to take it out of a product (1
// for other types).  An infinity is one in the first part alone, so products
// follow IEEE arithmetic.
template <int DT, int N>
__device__ __forceinline__ float to_operands(const Raw<DT> (&r)[N], Operand<DT> (&o)[N])
{
    if constexpr (DT == BCONV_F32) {
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(__uint_as_float(r[s].v[i >> 2][i & 3])));
        const uint32_t bits = lane_groups_max_bits(__float_as_uint(top));
        const Range<14> range(bits);
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h, l;
                split_pair(__uint_as_float(r[s].v[i >> 1][2 * (i & 1)]), __uint_as_float(r[s].v[i >> 1][2 * (i & 1) + 1]),
                           range.to, h, l);
                o[s].part[0][i] = h;
                o[s].part[1][i] = l;
            }
        if (__any(bits >= 0x7f800000u)) {
            // the second part of an infinity (infinity - infinity) becomes 0
#pragma unroll
            for (int s = 0; s < N; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t h = o[s].part[0][i];
                    if ((h & 0x7fffu) == 0x7c00u) o[s].part[1][i] &= 0xffff0000u;
                    if ((h & 0x7fff0000u) == 0x7c000000u) o[s].part[1][i] &= 0xffffu;
                }
        }
        return range.from;
    } else {
#pragma unroll
        for (int s = 0; s < N; ++s) o[s].part[0] = r[s].v[0];
        return 1.0f;
    }
}

template <int DT> __device__ __forceinline__ typename Elem<DT>::type round_to(float x)
{
    return static_cast<typename Elem<DT>::type>(x);
}

// Codes to operands.  A stored word holds 8 codes of consecutive k, code 2e at
// nibble e and code 2e+1 at nibble 4+e, rotated left by 3, so rotating right
// by 4e brings codes 2e and 2e+1 to bits 3..6 of the two halves, the top four
// of a bf16's seven mantissa bits: or-ing in the exponent of 2^-8 gives (16 + c)
// 2^-12.  Seven instructions for eight codes.  The same bits in fp16 (ten mantissa
// bits) under the exponent of 128 give 128 + c.
//
// What is left of the offset:
//   bf16: 16 (the products are exact; the caller takes 16 * sum x out).  Products
//         and what is made of them are in units of kUnit = 2^-12, so that no sum
//         over a group (at most 128 terms of 31 x each) passes the largest x, and
//         finite rows keep finite sums; nothing is lost at the other end, since
//         the matrix cores keep subnormal numbers;
//   fp16 and fp32: none: a packed subtraction of `zero` leaves the integer
//         itself, so that no cancellation costs bits.
constexpr uint32_t kCodeMask = 0x00780078u;
template <int DT> constexpr float kUnit = DT == BCONV_BF16 ? 1.0f / 4096.0f : 1.0f;
constexpr uint32_t kBase16 = 0x3b803b80u;   // bf16 2^-8, 2^-8: 16 units
constexpr uint32_t kBase128 = 0x58005800u;  // fp16 128, 128

__device__ __forceinline__ uint32_t rotr(uint32_t w, int n)
{
    return __builtin_amdgcn_alignbit(w, w, n);
}

// `zero` is subtracted from fp16 codes as a pair of halves holding 128 + zero.
template <int DT> struct Zero {
    f16x2 v;
    __device__ __forceinline__ explicit Zero(int z)
    {
        const _Float16 h = static_cast<_Float16>(128 + z);
        v = f16x2{h, h};
    }
};
template <> struct Zero<BCONV_BF16> {
    __device__ __forceinline__ explicit Zero(int) {}
};

// (x & mask) | base is one v_and_or_b32 when one constant is in a scalar
// register and the other in a vector register (as 32-bit literals they would
// take two instructions), so both are made opaque here, once a kernel.  The
// asm is empty on purpose: the compiler writes the registers itself and so
// keeps the wait states that a write next to a matrix instruction needs.
struct CodeBits {
    uint32_t mask, base;
    __device__ __forceinline__ uint32_t operator()(uint32_t t) const { return (t & mask) | base; }
};
__device__ __forceinline__ CodeBits opaque_bits(uint32_t mask, uint32_t base)
{
    asm("" : "+s"(mask));
    asm("" : "+v"(base));
    return CodeBits{mask, base};
}
template <int DT> __device__ __forceinline__ CodeBits code_bits()
{
    return opaque_bits(kCodeMask, DT == BCONV_BF16 ? kBase16 : kBase128);
}

template <int DT> __device__ __forceinline__ u32x4 decode(uint32_t w, const Zero<DT> &zero, const CodeBits &bits)
{
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // only the last pair wraps around; a plain shift issues twice as fast
        const uint32_t c = bits(e == 0 ? w : e < 3 ? w >> (4 * e) : rotr(w, 12));
        if constexpr (DT == BCONV_BF16) r[e] = c;
        else r[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, c) - zero.v);
    }
    return r;
}

// The constant operand of value v (in bf16 or, other types, fp16) in every position.
template <int DT> __device__ __forceinline__ u32x4 constant(float v)
{
    const uint16_t h = DT == BCONV_BF16 ? (uint16_t)(__float_as_uint(v) >> 16) : __builtin_bit_cast(uint16_t, (_Float16)v);
    const uint32_t w = h | ((uint32_t)h << 16);
    return u32x4{w, w, w, w};
}

}  // namespace bconv
