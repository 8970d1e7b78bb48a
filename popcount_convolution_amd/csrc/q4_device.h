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

// 16-byte matrix-core operands an fp32 value takes: three bf16 parts hold its
// 24 significant bits exactly; 16-bit types are operands as they are.
template <int DT> constexpr int kSplit = DT == BCONV_F32 ? 3 : 1;

// One lane's operand of v_mfma_f32_16x16x32: 8 consecutive k of one row or
// column, for each part of the split.
template <int DT> struct Operand {
    u32x4 part[kSplit<DT>];
};

template <int DT> __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT == BCONV_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

template <int DT> __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (DT == BCONV_F16)
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

__device__ __forceinline__ uint32_t pack_hi16(uint32_t lo, uint32_t hi)
{
    // bytes 2,3 of lo, then bytes 2,3 of hi
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// Three bf16 parts of x, by truncation: their sum is x exactly (8 significant
// bits each).  An infinity or NaN sits in the first part alone.
__device__ __forceinline__ void split3(float x, uint32_t &h, uint32_t &m, uint32_t &l)
{
    const uint32_t u = __float_as_uint(x);
    const bool finite = __builtin_isfinite(x);
    // a NaN whose bits all sit below the first part must not become an infinity
    h = x != x ? 0x7fc00000u : u & 0xffff0000u;
    const float r = finite ? x - __uint_as_float(h) : 0.0f;
    m = __float_as_uint(r) & 0xffff0000u;
    l = __float_as_uint(r - __uint_as_float(m));
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

template <int DT> __device__ __forceinline__ Operand<DT> to_operand(const Raw<DT> &r)
{
    Operand<DT> o;
    if constexpr (DT == BCONV_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h0, m0, l0, h1, m1, l1;
            split3(__uint_as_float(r.v[i >> 1][2 * (i & 1)]), h0, m0, l0);
            split3(__uint_as_float(r.v[i >> 1][2 * (i & 1) + 1]), h1, m1, l1);
            o.part[0][i] = pack_hi16(h0, h1);
            o.part[1][i] = pack_hi16(m0, m1);
            o.part[2][i] = pack_hi16(l0, l1);
        }
    } else {
        o.part[0] = r.v[0];
    }
    return o;
}

// 8 consecutive elements at p (offset k of a row of length len) as an operand;
// elements at or past len are 0.  `vec`: p is 16-byte aligned for k % 8 == 0.
template <int DT>
__device__ __forceinline__ Operand<DT> load_operand(const typename Elem<DT>::type *p, int k, int len, bool vec)
{
    return to_operand<DT>(vec && k + 8 <= len ? load_raw<DT>(p) : load_raw_masked<DT>(p, k, len));
}

template <int DT> __device__ __forceinline__ typename Elem<DT>::type round_to(float x)
{
    return static_cast<typename Elem<DT>::type>(x);
}

// Codes to operands.  A stored word holds 8 codes of consecutive k, code 2e at
// nibble e and code 2e+1 at nibble 4+e, rotated left by 3, so rotating right
// by 4e brings codes 2e and 2e+1 to bits 3..6 of the two halves, the top four
// of a bf16's seven mantissa bits: or-ing in the exponent of 16 gives 16 + c.
// Seven instructions for eight codes.  The same bits in fp16 (ten mantissa
// bits) under the exponent of 128 give 128 + c.
//
// What is left of the offset:
//   bf16: 16 (the products are exact; the caller takes 16 * sum x out);
//   fp16: none: a packed subtraction of `zero` leaves the integer itself;
//   fp32: none, so that no cancellation costs bits: the codes are spread to
//         bytes, `zero` is taken off four at a time (a byte holds 128 + c - z
//         and never borrows; with the top bit flipped it is c - z, signed), and
//         each byte converts to an exact float, whose upper half is the bf16.
constexpr uint32_t kCodeMask = 0x00780078u;
constexpr uint32_t kBase16 = 0x41804180u;   // bf16 16, 16
constexpr uint32_t kBase128 = 0x58005800u;  // fp16 128, 128

__device__ __forceinline__ uint32_t rotr(uint32_t w, int n)
{
    return __builtin_amdgcn_alignbit(w, w, n);
}

// `zero` is subtracted from the codes where the type allows (see above): fp32
// takes it as four bytes of 128 - zero, fp16 as a pair of halves holding 128 + zero.
template <int DT> struct Zero;
template <> struct Zero<BCONV_BF16> {
    __device__ __forceinline__ explicit Zero(int) {}
};
template <> struct Zero<BCONV_F16> {
    f16x2 v;
    __device__ __forceinline__ explicit Zero(int z)
    {
        const _Float16 h = static_cast<_Float16>(128 + z);
        v = f16x2{h, h};
    }
};
template <> struct Zero<BCONV_F32> {
    uint32_t v;
    __device__ __forceinline__ explicit Zero(int z) : v((uint32_t)(128 - z) * 0x01010101u) {}
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
    return opaque_bits(kCodeMask, DT == BCONV_F16 ? kBase128 : kBase16);
}

template <int DT> __device__ __forceinline__ u32x4 decode(uint32_t w, const Zero<DT> &zero, const CodeBits &bits)
{
    u32x4 r;
    if constexpr (DT == BCONV_F32) {
        // nibbles (rotated by 3) at even and odd places: bytes b of `even` are
        // nibbles 2b, of `odd` nibbles 2b + 1; codes 2e, 2e + 1 are nibbles e, 4 + e
        const uint32_t even = ((rotr(w, 3) & 0x0f0f0f0fu) + zero.v) ^ 0x80808080u;
        const uint32_t odd = ((rotr(w, 7) & 0x0f0f0f0fu) + zero.v) ^ 0x80808080u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t src = e & 1 ? odd : even;
            const float lo = (float)(int8_t)(src >> (8 * (e >> 1))), hi = (float)(int8_t)(src >> (8 * (2 + (e >> 1))));
            r[e] = pack_hi16(__float_as_uint(lo), __float_as_uint(hi));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // only the last pair wraps around; a plain shift issues twice as fast
            const uint32_t c = bits(e == 0 ? w : e < 3 ? w >> (4 * e) : rotr(w, 12));
            if constexpr (DT == BCONV_F16) r[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, c) - zero.v);
            else r[e] = c;
        }
    }
    return r;
}

// The constant operand of bf16 value v in every position.
__device__ __forceinline__ u32x4 bf16_const(float v)
{
    const uint32_t h = __float_as_uint(v) >> 16, w = h | (h << 16);
    return u32x4{w, w, w, w};
}

}  // namespace bconv
