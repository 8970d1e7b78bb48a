// The write of new keys and values into the paged 4-bit cache, and the cache's
// geometry.
//
// Per group of channels: s = fp16((max - min) * fp32(1/15)), b = fp16(min + 8 s),
// c = clamp(rint((x - b) * (1 / s)) + 8, 0, 15).  Every operation is one fp32
// rounding (no contraction is possible in these forms, and 1 / s is the
// correctly rounded quotient), so the codes are a function of the values alone.
#include <hip/hip_runtime.h>

#include "kv4.h"

namespace bconv {

bconv_status_t kv4_geometry(const bconv_kv4_desc_t *d, Kv4Geom *g)
{
    if (!d) return fail(BCONV_ERR_INVALID_ARGUMENT, "desc is NULL");
    if (d->block_size < 16 || d->block_size > 1024 || (d->block_size & (d->block_size - 1)))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "block_size must be a power of two in [16, 1024]");
    if (d->num_blocks < 1 || (long long)d->num_blocks * d->block_size >= (1LL << 31))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "num_blocks must be >= 1 and num_blocks*block_size below 2^31");
    if (d->kv_heads < 1 || d->kv_heads > 1024)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "kv_heads must be in [1, 1024]");
    if (d->head_dim < 8 || d->head_dim > 256 || d->head_dim % 8)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of 8 in [8, 256]");
    if (d->group != 32 && d->group != 64 && d->group != 128)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "group must be 32, 64 or 128");
    g->num_blocks = d->num_blocks;
    g->block_shift = __builtin_ctz((unsigned)d->block_size);
    g->kv_heads = d->kv_heads;
    g->dim = d->head_dim;
    g->dim_padded = d->head_dim <= 64 ? 64 : d->head_dim <= 128 ? 128 : 256;
    g->groups = g->dim_padded <= d->group ? 1 : g->dim_padded / d->group;
    g->row_bytes = g->dim_padded / 2;
    g->v_codes = d->block_size * g->row_bytes;
    g->k_scales = 2 * g->v_codes;
    g->v_scales = g->k_scales + d->block_size * g->groups * 4;
    g->record_bytes = g->v_scales + d->block_size * g->groups * 4;
    return BCONV_OK;
}

struct AppendSide {
    const void *x;
    long long token_stride, head_stride;
    void *out;
    int vec;      // rows of x are 16-byte aligned
    int vec_out;  // rows of out are
};

struct AppendArgs {
    AppendSide side[2];
    char *pool;
    const int *slots;
    int tokens;
    Kv4Geom g;
    long long first_row;  // of the launch
};

// DP / 8 lanes a row (token, head, side), 8 channels a lane; since head_dim is
// a multiple of 8 a lane's channels are all real or all padding.  LG lanes
// share a group.  Bound by the bytes of x and of the values written back: 8193
// tokens of 8 heads of 128 channels in bf16, 76.6 MB with the values, 19.1 to 19.6 us
// (3.9 to 4.0 TB/s; a large copy reaches 4.77 to 5.16).  One decoding step of 32
// tokens is a launch (3.7 us by trace, 3.3 a call in a graph).
template <int DT, int DP, int LG>
__global__ __launch_bounds__(256) void kv4_append_kernel(AppendArgs a)
{
    typedef typename Elem<DT>::type T;
    constexpr int L = DP / 8;
    const int p = threadIdx.x % L;
    const bool is_v = blockIdx.y != 0;
    const AppendSide &side = a.side[is_v ? 1 : 0];
    const long long rows = (long long)a.tokens * a.g.kv_heads;
    const long long row = a.first_row + (long long)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool live = row < rows;  // every lane stays for the exchanges
    const int token = live ? (int)(row / a.g.kv_heads) : 0, head = live ? (int)(row % a.g.kv_heads) : 0;
    const bool real = live && 8 * p < a.g.dim;

    float x[8];
    float lo = __builtin_inff(), hi = -__builtin_inff();
    if (real) {
        const T *src = static_cast<const T *>(side.x) + token * side.token_stride + head * side.head_stride + 8 * p;
        if (side.vec) {
            if constexpr (DT == BCONV_F32) {
                const f32x4 u = *reinterpret_cast<const f32x4 *>(src), v = *reinterpret_cast<const f32x4 *>(src + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = u[i];
                    x[4 + i] = v[i];
                }
            } else {
                typedef T Tx8 __attribute__((ext_vector_type(8)));
                const Tx8 u = *reinterpret_cast<const Tx8 *>(src);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = (float)u[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)src[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = x[i] != x[i] ? 0.0f : fminf(fmaxf(x[i], -65504.0f), 65504.0f);
            lo = fminf(lo, x[i]);
            hi = fmaxf(hi, x[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    }
#pragma unroll
    for (int d = 1; d < LG; d *= 2) {
        lo = fminf(lo, __shfl_xor(lo, d));
        hi = fmaxf(hi, __shfl_xor(hi, d));
    }
    // a group of padding alone: lo > hi
    const bool any = lo <= hi;
    const _Float16 sh = (_Float16)(any ? (hi - lo) * (1.0f / 15.0f) : 0.0f);
    const float s = (float)sh;
    const _Float16 bh = (_Float16)(any ? lo + 8.0f * s : 0.0f);
    const float b = (float)bh;
    const float r = s > 0.0f ? 1.0f / s : 0.0f;
    uint32_t code[8], natural = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf((x[i] - b) * r) + 8.0f, 0.0f), 15.0f);
        code[i] = real ? (uint32_t)c : 8u;
        natural |= code[i] << (4 * i);
    }

    // the values that the cache stands for
    if (side.out && real) {
        T *dst = static_cast<T *>(side.out) + row * a.g.dim + 8 * p;
        if (side.vec_out) {
            if constexpr (DT == BCONV_F32) {
                f32x4 u, v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = __builtin_fmaf(s, (float)code[i] - 8.0f, b);
                    v[i] = __builtin_fmaf(s, (float)code[4 + i] - 8.0f, b);
                }
                *reinterpret_cast<f32x4 *>(dst) = u;
                *reinterpret_cast<f32x4 *>(dst + 4) = v;
            } else {
                typedef T Tx8 __attribute__((ext_vector_type(8)));
                Tx8 u;
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = round_to<DT>(__builtin_fmaf(s, (float)code[i] - 8.0f, b));
                *reinterpret_cast<Tx8 *>(dst) = u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = round_to<DT>(__builtin_fmaf(s, (float)code[i] - 8.0f, b));
        }
    }

    uint32_t word;
    int at;
    if (!is_v) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) w |= (code[2 * e] << (4 * e)) | (code[2 * e + 1] << (16 + 4 * e));
        word = (w << 3) | (w >> 29);
        at = (p & 3) * (DP / 32) + (p >> 2);
    } else {
        // nibble n of word p is nibble j of part r, channel 16 j + r, which
        // lane 2 j + r / 8 of the row holds
        const int base = (threadIdx.x & 63) - p;
        word = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int q = 8 * p + n, r2 = q / (DP / 16), j = q % (DP / 16);
            const uint32_t w = (uint32_t)__shfl((int)natural, base + 2 * j + (r2 >> 3));
            word |= ((w >> (4 * (r2 & 7))) & 15u) << (4 * n);
        }
        at = p;
    }
    if (!live) return;
    const int slot = a.slots[token];
    const int block = slot >> a.g.block_shift;
    if (slot < 0 || block >= a.g.num_blocks) return;
    char *rec = a.pool + ((long long)block * a.g.kv_heads + head) * a.g.record_bytes;
    const int t = slot & ((1 << a.g.block_shift) - 1);
    reinterpret_cast<uint32_t *>(rec + (is_v ? a.g.v_codes : 0) + t * (DP / 2))[at] = word;
    if (p % LG == 0) {
        const uint32_t sb =
            (uint32_t)__builtin_bit_cast(uint16_t, sh) | ((uint32_t)__builtin_bit_cast(uint16_t, bh) << 16);
        reinterpret_cast<uint32_t *>(rec + (is_v ? a.g.v_scales : a.g.k_scales))[t * a.g.groups + p / LG] = sb;
    }
}

template <int DT, int DP>
hipError_t launch_append_dim(AppendArgs a, int group, hipStream_t s)
{
    constexpr int ROWS = 256 / (DP / 8);  // a workgroup
    const long long rows = (long long)a.tokens * a.g.kv_heads;
    const int lanes = (group < DP ? group : DP) / 8;
    return launch_slices((rows + ROWS - 1) / ROWS, [&](long long first, unsigned count) {
        a.first_row = first * ROWS;
        const dim3 grid(count, 2);
        if (lanes == 4)
            hipLaunchKernelGGL((kv4_append_kernel<DT, DP, 4>), grid, dim3(256), 0, s, a);
        else if (lanes == 8)
            hipLaunchKernelGGL((kv4_append_kernel<DT, DP, 8>), grid, dim3(256), 0, s, a);
        else if constexpr (DP >= 128)
            hipLaunchKernelGGL((kv4_append_kernel<DT, DP, 16>), grid, dim3(256), 0, s, a);
    });
}

template <int DT>
hipError_t launch_append(const AppendArgs &a, int group, hipStream_t s)
{
    switch (a.g.dim_padded) {
    case 64: return launch_append_dim<DT, 64>(a, group, s);
    case 128: return launch_append_dim<DT, 128>(a, group, s);
    default: return launch_append_dim<DT, 256>(a, group, s);
    }
}

}  // namespace bconv

using bconv::fail;

extern "C" {

bconv_status_t bconv_kv4_layout(const bconv_kv4_desc_t *desc, bconv_kv4_layout_t *layout)
{
    if (!layout) return fail(BCONV_ERR_INVALID_ARGUMENT, "layout is NULL");
    bconv::Kv4Geom g;
    const bconv_status_t st = bconv::kv4_geometry(desc, &g);
    if (st != BCONV_OK) return st;
    *layout = bconv_kv4_layout_t{};
    layout->record_bytes = (size_t)g.record_bytes;
    layout->pool_bytes = (size_t)g.record_bytes * g.kv_heads * g.num_blocks;
    layout->row_bytes = g.row_bytes;
    layout->dim_padded = g.dim_padded;
    layout->groups = g.groups;
    layout->v_codes_offset = (size_t)g.v_codes;
    layout->k_scales_offset = (size_t)g.k_scales;
    layout->v_scales_offset = (size_t)g.v_scales;
    return BCONV_OK;
}

bconv_status_t bconv_kv4_append(const bconv_kv4_desc_t *desc, void *stream, void *pool, int32_t tokens, int32_t dtype,
                                const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots, void *k_out,
                                void *v_out)
{
    bconv::AppendArgs a{};
    const bconv_status_t st = bconv::kv4_geometry(desc, &a.g);
    if (st != BCONV_OK) return st;
    if (tokens < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "tokens must be >= 0");
    const int es = bconv::dtype_size(dtype);
    if (!es) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
    if (tokens == 0) return BCONV_OK;
    if (!pool || !k || !v || !slots) return fail(BCONV_ERR_INVALID_ARGUMENT, "pool, k, v and slots must not be NULL");
    if ((uintptr_t)pool % 16) return fail(BCONV_ERR_INVALID_ARGUMENT, "the pool must be 16-byte aligned");
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)k_out | (uintptr_t)v_out) % es || (uintptr_t)slots % 4)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "a tensor is not aligned to its element");
    const int64_t strides[] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    for (const int64_t t : strides)
        if (t < 0 || t > (1LL << 40)) return fail(BCONV_ERR_INVALID_ARGUMENT, "strides must be in [0, 2^40]");
    if ((long long)tokens * a.g.kv_heads >= (1LL << 31))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "tokens*kv_heads must stay below 2^31");
    a.pool = static_cast<char *>(pool);
    a.slots = slots;
    a.tokens = tokens;
    const void *x[2] = {k, v};
    void *out[2] = {k_out, v_out};
    for (int i = 0; i < 2; ++i) {
        a.side[i] = {x[i], strides[2 * i], strides[2 * i + 1], out[i],
                     (uintptr_t)x[i] % 16 == 0 && strides[2 * i] * es % 16 == 0 && strides[2 * i + 1] * es % 16 == 0,
                     (uintptr_t)out[i] % 16 == 0};
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    switch (dtype) {
    case BCONV_F32: e = bconv::launch_append<BCONV_F32>(a, desc->group, s); break;
    case BCONV_F16: e = bconv::launch_append<BCONV_F16>(a, desc->group, s); break;
    default: e = bconv::launch_append<BCONV_BF16>(a, desc->group, s); break;
    }
    if (e != hipSuccess) return bconv::hip_fail(e, "cache append kernel");
    return BCONV_OK;
}

}  // extern "C"
