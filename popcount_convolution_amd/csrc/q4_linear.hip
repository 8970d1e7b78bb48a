// Linear layers with 4-bit weights and group scales.
//
//   y[m][o] = bias[o] + sum_g s[o][g] * (sum_{k in g} x[m][k] c[o][k] - z[o][g] sum_{k in g} x[m][k])
//
// Outputs are the rows and x rows the columns of v_mfma_f32_16x16x32 products,
// so that up to 16 rows of x cost one matrix instruction per 16 x 32 codes and
// the codes go from global memory to registers to the matrix cores without
// passing LDS.  Weights are laid out once, at create, in the order the lanes
// read them: one 16-byte load a lane is 16 outputs x 128 inputs.
#include <hip/hip_runtime.h>

#include <cstring>
#include <new>

#include "host.h"
#include "q4_device.h"

namespace bconv {

constexpr int kChunk = 128;         // inputs of one 16-byte load a lane
constexpr int kFewWaves = 8;        // waves that split the inputs of one output tile
constexpr int kGroupsMax = kChunk / 32;

struct Q4Args {
    const uint32_t *codes;   // [tiles][chunks][64 lanes][4]
    const uint16_t *scales;  // fp16 [tiles][chunks][groups a chunk][16]
    const uint8_t *zeros;    // [tiles][chunks][groups a chunk][16] or nullptr
    const float *bias;       // [n] or nullptr
    const void *x;
    void *y;
    long long ldx, ldy;
    int m, n, k;
    int tiles, chunks;
    int vec;                 // rows of x are 16-byte aligned
};

// Weights in lane order.  Word s of lane (row r = lane & 15, lg = lane >> 4) of
// a chunk is inputs 128 chunk + 32 s + 8 lg .. +7 of output 16 tile + r, i.e.
// one user word, its nibbles reordered for decode().
__global__ void q4_prepack_kernel(const uint32_t *user, uint32_t *codes, int n, int k, int tiles, int chunks)
{
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)tiles * chunks * 256) return;
    const int s = (int)(i & 3), lane = (int)(i >> 2) & 63;
    const long long tc = i >> 8;
    const int chunk = (int)(tc % chunks), tile = (int)(tc / chunks);
    const int o = tile * 16 + (lane & 15), k0 = chunk * kChunk + s * 32 + (lane >> 4) * 8;
    uint32_t w = 0;
    if (o < n && k0 < k) {
        w = user[(long long)o * ((k + 7) / 8) + k0 / 8];
        if (k - k0 < 8) w &= (1u << (4 * (k - k0))) - 1u;
    }
    uint32_t r = 0;
    for (int e = 0; e < 4; ++e) {
        r |= ((w >> (8 * e)) & 15u) << (4 * e);
        r |= ((w >> (8 * e + 4)) & 15u) << (16 + 4 * e);
    }
    codes[i] = (r << 3) | (r >> 29);
}

// Scales and zero points in [tile][chunk][group][16 outputs] order; padding
// has scale 0.
__global__ void q4_prepack_scales_kernel(const uint16_t *user_s, const uint8_t *user_z, uint16_t *scales, uint8_t *zeros,
                                         int n, int groups, int per_chunk, int tiles, int chunks)
{
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)tiles * chunks * per_chunk * 16) return;
    const int r = (int)(i & 15);
    long long j = i >> 4;
    const int g = (int)(j % per_chunk);
    j /= per_chunk;
    const int chunk = (int)(j % chunks), tile = (int)(j / chunks);
    const int o = tile * 16 + r, group = chunk * per_chunk + g;
    const bool in = o < n && group < groups;
    scales[i] = in ? user_s[(long long)o * groups + group] : 0;
    if (zeros) zeros[i] = in ? user_z[(long long)o * groups + group] : 8;
}

// One chunk (16 RT outputs x 128 inputs) times NT tiles of 16 rows of x, added
// to acc.  STEPS: 32-input steps a group.  Per group and output tile the exact
// products of one group are summed first, then scaled once in fp32.
template <int DT, bool ZP, int STEPS, int RT, int NT>
__device__ __forceinline__ void chunk_product(const u32x4 (&w)[RT], const Operand<DT> (&xf)[4][NT],
                                              const uint16_t *const (&sc)[RT], const uint8_t *const (&zp)[RT], int lane,
                                              f32x4 (&acc)[RT][NT])
{
    const int row = lane & 15, lg = lane >> 4;
#pragma unroll
    for (int g = 0; g < 4 / STEPS; ++g) {
        // bf16: the offset 16 + z of the codes leaves -(16 + z) sum x, on the
        // matrix cores as well (a constant operand times x)
        f32x4 off[NT];
        if constexpr (DT == BCONV_BF16) {
            const u32x4 c = bf16_const(ZP ? -1.0f : -24.0f);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                off[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s) off[t] = mfma_parts<DT>(c, xf[g * STEPS + s][t], off[t]);
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
            const f16x4 s4 = *reinterpret_cast<const f16x4 *>(sc[r] + g * 16 + lg * 4);
            int z = 8;
            uint32_t z4 = 0;
            if constexpr (ZP) {
                if constexpr (DT == BCONV_BF16)
                    z4 = *reinterpret_cast<const uint32_t *>(zp[r] + g * 16 + lg * 4);
                else
                    z = zp[r][g * 16 + row];
            }
            const Zero<DT> zero(z);
            f32x4 d[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if constexpr (DT == BCONV_BF16) {
                    if constexpr (ZP) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[t][i] = (float)(16 + ((z4 >> (8 * i)) & 255u)) * off[t][i];
                    } else {
                        d[t] = off[t];
                    }
                } else {
                    d[t] = f32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const u32x4 a = decode<DT>(w[r][g * STEPS + s], zero);
#pragma unroll
                for (int t = 0; t < NT; ++t) d[t] = mfma_parts<DT>(a, xf[g * STEPS + s][t], d[t]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf((float)s4[i], d[t][i], acc[r][t][i]);
        }
    }
}

// Few rows of x.  A workgroup takes 16 RT outputs and 16 NT rows of x; its
// waves split the inputs chunk by chunk and add their sums in LDS, in a fixed
// order.
template <int DT, bool ZP, int STEPS, int RT, int NT>
__global__ __launch_bounds__(kFewWaves * 64) void q4_few_kernel(Q4Args a)
{
    typedef typename Elem<DT>::type T;
    __shared__ f32x4 part[kFewWaves][RT * NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tile0 = blockIdx.x * RT, m0 = blockIdx.y * 16 * NT;
    const int row = lane & 15, lg = lane >> 4;
    constexpr int per_chunk = 4 / STEPS;

    f32x4 acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};

    for (int c = wave; c < a.chunks; c += kFewWaves) {
        u32x4 w[RT];
        const uint16_t *sc[RT];
        const uint8_t *zp[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int tile = tile0 + r < a.tiles ? tile0 + r : a.tiles - 1;
            const long long tc = (long long)tile * a.chunks + c;
            w[r] = *reinterpret_cast<const u32x4 *>(a.codes + tc * 256 + lane * 4);
            sc[r] = a.scales + tc * per_chunk * 16;
            zp[r] = ZP ? a.zeros + tc * per_chunk * 16 : nullptr;
        }
        Operand<DT> xf[4][NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int m = m0 + t * 16 + row;
            const T *xr = static_cast<const T *>(a.x) + (long long)m * a.ldx;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = c * kChunk + s * 32 + lg * 8;
                if (m < a.m && k < a.k) {
                    xf[s][t] = load_operand<DT>(xr + k, k, a.k, a.vec != 0);
                } else {
#pragma unroll
                    for (int p = 0; p < kSplit<DT>; ++p) xf[s][t].part[p] = u32x4{0, 0, 0, 0};
                }
            }
        }
        chunk_product<DT, ZP, STEPS, RT, NT>(w, xf, sc, zp, lane, acc);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[wave][r * NT + t][lane] = acc[r][t];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * NT * 64; e += kFewWaves * 64) {
        const int l = e & 63, rt = e >> 6;
        const int m = m0 + (rt % NT) * 16 + (l & 15);
        const int o0 = (tile0 + rt / NT) * 16 + (l >> 4) * 4;
        if (m >= a.m || o0 >= a.n) continue;
        f32x4 v = part[0][rt][l];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += part[w][rt][l];
        T *y = static_cast<T *>(a.y) + (long long)m * a.ldy + o0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (o0 + i < a.n) y[i] = round_to<DT>(v[i] + (a.bias ? a.bias[o0 + i] : 0.0f));
    }
}

template <int DT, bool ZP, int STEPS, int RT, int NT>
hipError_t run_few(const Q4Args &a, hipStream_t s)
{
    const dim3 grid((a.tiles + RT - 1) / RT, (a.m + 16 * NT - 1) / (16 * NT));
    hipLaunchKernelGGL((q4_few_kernel<DT, ZP, STEPS, RT, NT>), grid, dim3(kFewWaves * 64), 0, s, a);
    return hipGetLastError();
}

template <int DT, bool ZP, int STEPS>
hipError_t run_linear(const Q4Args &a, hipStream_t s)
{
    return run_few<DT, ZP, STEPS, 1, 1>(a, s);
}

template <int DT, bool ZP>
hipError_t dispatch_group(const Q4Args &a, int group, hipStream_t s)
{
    switch (group) {
    case 32: return run_linear<DT, ZP, 1>(a, s);
    case 64: return run_linear<DT, ZP, 2>(a, s);
    default: return run_linear<DT, ZP, 4>(a, s);
    }
}

template <int DT>
hipError_t dispatch_zero(const Q4Args &a, int group, hipStream_t s)
{
    return a.zeros ? dispatch_group<DT, true>(a, group, s) : dispatch_group<DT, false>(a, group, s);
}

}  // namespace bconv

struct bconv_q4_linear {
    bconv_q4_linear_desc_t desc;
    int device;
    int tiles, chunks, per_chunk;
    uint32_t *d_codes;
    uint16_t *d_scales;
    uint8_t *d_zeros;
    float *d_bias;
};

namespace {

using bconv::DeviceGuard;
using bconv::fail;
using bconv::hip_fail;
using bconv::ranges_overlap;
using bconv::upload;

constexpr int32_t kMaxFeatures = 1 << 20;

bconv_status_t check_desc(const bconv_q4_linear_desc_t *d)
{
    if (!d) return fail(BCONV_ERR_INVALID_ARGUMENT, "desc is NULL");
    if (d->in_features < 1 || d->in_features > kMaxFeatures || d->out_features < 1 || d->out_features > kMaxFeatures)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "in_features/out_features must be in [1, %d]", kMaxFeatures);
    if ((long long)d->in_features * d->out_features > (1LL << 34))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "in_features*out_features exceeds 2^34");
    if (d->group != 32 && d->group != 64 && d->group != 128)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "group must be 32, 64 or 128");
    return BCONV_OK;
}

void release(bconv_q4_linear *h)
{
    void *ptrs[] = {h->d_codes, h->d_scales, h->d_zeros, h->d_bias};
    for (void *p : ptrs)
        if (p) (void)hipFree(p);
    delete h;
}

int dtype_bytes(int32_t dtype)
{
    return dtype == BCONV_F32 ? 4 : dtype == BCONV_F16 || dtype == BCONV_BF16 ? 2 : 0;
}

template <typename T> bconv_status_t device_alloc(T **p, size_t count)
{
    const hipError_t e = hipMalloc(reinterpret_cast<void **>(p), count * sizeof(T));
    if (e == hipSuccess) return BCONV_OK;
    *p = nullptr;
    return fail(BCONV_ERR_ALLOC, "hipMalloc(%zu): %s", count * sizeof(T), hipGetErrorString(e));
}

}  // namespace

extern "C" {

bconv_status_t bconv_q4_linear_create(const bconv_q4_linear_desc_t *desc, const uint32_t *weight_words,
                                      const uint16_t *scales, const uint8_t *zeros, const float *bias,
                                      bconv_q4_linear_t *out)
{
    if (!out) return fail(BCONV_ERR_INVALID_ARGUMENT, "out is NULL");
    *out = nullptr;
    bconv_status_t st = check_desc(desc);
    if (st != BCONV_OK) return st;
    if (!weight_words || !scales) return fail(BCONV_ERR_INVALID_ARGUMENT, "weight_words or scales is NULL");
    const int n = desc->out_features, k = desc->in_features, groups = (k + desc->group - 1) / desc->group;
    if (zeros)
        for (size_t i = 0; i < (size_t)n * groups; ++i)
            if (zeros[i] > 15) return fail(BCONV_ERR_INVALID_ARGUMENT, "zeros[%zu] = %d is not in [0, 15]", i, zeros[i]);

    bconv_q4_linear *h = new (std::nothrow) bconv_q4_linear();
    if (!h) return fail(BCONV_ERR_ALLOC, "host allocation failed");
    h->desc = *desc;
    h->tiles = (n + 15) / 16;
    h->chunks = (k + bconv::kChunk - 1) / bconv::kChunk;
    h->per_chunk = bconv::kChunk / desc->group;
    hipError_t e = hipGetDevice(&h->device);
    if (e != hipSuccess) {
        release(h);
        return hip_fail(e, "hipGetDevice");
    }
    uint32_t *d_words = nullptr;
    uint16_t *d_s = nullptr;
    uint8_t *d_z = nullptr;
    const size_t nc = (size_t)h->tiles * h->chunks * 256, ns = (size_t)h->tiles * h->chunks * h->per_chunk * 16;
    if ((st = upload(weight_words, (size_t)n * ((k + 7) / 8), &d_words)) == BCONV_OK &&
        (st = upload(scales, (size_t)n * groups, &d_s)) == BCONV_OK &&
        (st = upload(zeros, (size_t)n * groups, &d_z)) == BCONV_OK &&
        (st = upload(bias, (size_t)n, &h->d_bias)) == BCONV_OK &&
        (st = device_alloc(&h->d_codes, nc)) == BCONV_OK && (st = device_alloc(&h->d_scales, ns)) == BCONV_OK &&
        (!zeros || (st = device_alloc(&h->d_zeros, ns)) == BCONV_OK)) {
        hipLaunchKernelGGL(bconv::q4_prepack_kernel, dim3((unsigned)((nc + 255) / 256)), dim3(256), 0, nullptr, d_words,
                           h->d_codes, n, k, h->tiles, h->chunks);
        hipLaunchKernelGGL(bconv::q4_prepack_scales_kernel, dim3((unsigned)((ns + 255) / 256)), dim3(256), 0, nullptr,
                           d_s, d_z, h->d_scales, h->d_zeros, n, groups, h->per_chunk, h->tiles, h->chunks);
        e = hipGetLastError();
        if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
        if (e != hipSuccess) st = hip_fail(e, "weight prepack");
    }
    void *tmp[] = {d_words, d_s, d_z};
    for (void *p : tmp)
        if (p) (void)hipFree(p);
    if (st != BCONV_OK) {
        release(h);
        return st;
    }
    *out = h;
    return BCONV_OK;
}

bconv_status_t bconv_q4_linear_workspace_size(bconv_q4_linear_t h, int32_t rows, int32_t dtype, size_t *bytes)
{
    if (!h || !bytes) return fail(BCONV_ERR_INVALID_ARGUMENT, "handle or bytes is NULL");
    if (rows < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows must be >= 0");
    if (!dtype_bytes(dtype)) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
    *bytes = 0;
    return BCONV_OK;
}

bconv_status_t bconv_q4_linear_forward(bconv_q4_linear_t h, void *stream, int32_t rows, int32_t dtype, const void *x,
                                       int64_t ldx, void *y, int64_t ldy, void *workspace, size_t workspace_bytes)
{
    if (!h) return fail(BCONV_ERR_INVALID_ARGUMENT, "handle is NULL");
    if (rows < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows must be >= 0");
    const int es = dtype_bytes(dtype);
    if (!es) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
    if (rows == 0) return BCONV_OK;
    const int n = h->desc.out_features, k = h->desc.in_features;
    if (!x || !y) return fail(BCONV_ERR_INVALID_ARGUMENT, "x/y must not be NULL");
    if (ldx < k || ldy < n) return fail(BCONV_ERR_INVALID_ARGUMENT, "ldx/ldy shorter than a row");
    if (ldx > (1LL << 40) || ldy > (1LL << 40)) return fail(BCONV_ERR_INVALID_ARGUMENT, "ldx/ldy too large");
    if (((uintptr_t)x | (uintptr_t)y) % es) return fail(BCONV_ERR_INVALID_ARGUMENT, "x/y not aligned to an element");
    const size_t xb = ((size_t)(rows - 1) * ldx + k) * es, yb = ((size_t)(rows - 1) * ldy + n) * es;
    if (ranges_overlap(x, xb, y, yb)) return fail(BCONV_ERR_INVALID_ARGUMENT, "x and y overlap");
    size_t need = 0;
    bconv_status_t st = bconv_q4_linear_workspace_size(h, rows, dtype, &need);
    if (st != BCONV_OK) return st;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(BCONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                    workspace ? workspace_bytes : (size_t)0);

    DeviceGuard guard(h->device);
    if (guard.err != hipSuccess) return hip_fail(guard.err, "hipSetDevice");
    bconv::Q4Args a{};
    a.codes = h->d_codes;
    a.scales = h->d_scales;
    a.zeros = h->d_zeros;
    a.bias = h->d_bias;
    a.x = x;
    a.y = y;
    a.ldx = ldx;
    a.ldy = ldy;
    a.m = rows;
    a.n = n;
    a.k = k;
    a.tiles = h->tiles;
    a.chunks = h->chunks;
    a.vec = ((uintptr_t)x % 16 == 0) && (ldx * es % 16 == 0);
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    switch (dtype) {
    case BCONV_F32: e = bconv::dispatch_zero<BCONV_F32>(a, h->desc.group, s); break;
    case BCONV_F16: e = bconv::dispatch_zero<BCONV_F16>(a, h->desc.group, s); break;
    default: e = bconv::dispatch_zero<BCONV_BF16>(a, h->desc.group, s); break;
    }
    if (e != hipSuccess) return hip_fail(e, "4-bit linear kernel");
    return BCONV_OK;
}

bconv_status_t bconv_q4_linear_destroy(bconv_q4_linear_t h)
{
    if (!h) return BCONV_OK;
    DeviceGuard guard(h->device);
    release(h);
    return BCONV_OK;
}

}  // extern "C"
