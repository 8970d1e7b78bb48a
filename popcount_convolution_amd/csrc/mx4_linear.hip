// Linear layers of microscaled 4-bit floats, one or one for each expert.
//
//   y[i][o] = bias[f][o] + sum_k Q(x[r])[k] W[f][o][k]
//
// Outputs are the rows and rows of x the columns of
// v_mfma_scale_f32_16x16x128_f8f6f4 products, which take the codes and the powers
// of two as they are held.  Weights are laid out once, at create, in the order
// the lanes read them: one 16-byte load a lane is 16 outputs x 128 inputs.
#include <hip/hip_runtime.h>

#include <new>

#include "host.h"
#include "mx4.h"

namespace bconv {

// A layer's weights: [experts][tiles][steps][2][64 lanes][16 bytes], scales
// [experts][tiles][steps][64 lanes][2 bytes].
struct Mx4Args {
    const u32x4 *codes;
    const uint16_t *scales;
    const float *bias;       // [experts][n] or nullptr
    const void *x;           // elements, or nullptr
    const uint8_t *xc, *xs;  // quantised rows
    void *y;
    const int *offsets, *order;
    long long ldx, ldy;
    int rows, x_rows, choices;
    int n, k, tiles, steps, experts;
};

// 8 codes (word j of 16 bytes) of lane (r, lg), instruction i of a step: values
// 32 b + 8 j .. of row r, b = 8 step + 2 lg + i.
__global__ void mx4_prepack_kernel(const uint8_t *user, uint32_t *codes, int n, int k, int tiles, int steps, long long first,
                                   long long total)
{
    long long id = first + (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= total) return;
    uint32_t *to = codes + id;
    const int j = (int)(id & 3), lane = (int)(id >> 2) & 63, i = (int)(id >> 8) & 1;
    id >>= 9;
    const int step = (int)(id % steps);
    id /= steps;
    const int tile = (int)(id % tiles);
    const long long f = id / tiles;
    const int o = tile * 16 + (lane & 15), k0 = step * kStep + (lane >> 4) * 64 + i * 32 + j * 8;
    uint32_t w = 0;
    if (o < n) {
        const uint8_t *row = user + (f * n + o) * ((k + 1) / 2);
        for (int v = 0; v < 4; ++v) {
            uint32_t b = k0 + 2 * v < k ? row[k0 / 2 + v] : 0u;
            if (k0 + 2 * v + 1 >= k) b &= 15u;
            w |= b << (8 * v);
        }
    }
    *to = w;
}

__global__ void mx4_prepack_scales_kernel(const uint8_t *user, uint8_t *scales, int n, int k, int tiles, int steps, long long first,
                                          long long total)
{
    long long id = first + (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= total) return;
    uint8_t *to = scales + id;
    const int i = (int)(id & 1), lane = (int)(id >> 1) & 63;
    id >>= 7;
    const int step = (int)(id % steps);
    id /= steps;
    const int tile = (int)(id % tiles);
    const long long f = id / tiles;
    const int o = tile * 16 + (lane & 15), b = step * (kStep / 32) + (lane >> 4) * 2 + i, blocks = (k + 31) / 32;
    *to = o < n && b < blocks ? user[(f * n + o) * blocks + b] : 0;
}

// Result rows [begin, end) of expert f; of f = experts: those of none.
struct Span {
    int begin, end;
};

__device__ __forceinline__ int clamped_offset(const Mx4Args &a, int f)
{
    const int o = a.offsets[f];
    return o < 0 ? 0 : o > a.rows ? a.rows : o;
}

__device__ __forceinline__ Span expert_span(const Mx4Args &a, int f)
{
    if (!a.offsets) return {0, a.rows};
    return {clamped_offset(a, f), f < a.experts ? clamped_offset(a, f + 1) : a.rows};
}

// Input row of result row i (i < rows).
__device__ __forceinline__ int input_row(const Mx4Args &a, int i)
{
    if (a.choices == 0) return i;
    const int p = a.order[i];
    const int r = p < 0 ? 0 : p / a.choices;
    return r < a.x_rows ? r : a.x_rows - 1;
}

// 4 consecutive outputs of result row i, with the bias, as far as there are outputs.
template <int DT> __device__ __forceinline__ void store_four(const Mx4Args &a, int f, int i, int o0, f32x4 v)
{
    typedef typename Elem<DT>::type T;
    T *y = static_cast<T *>(a.y) + (long long)i * a.ldy + o0;
    const float *b = a.bias ? a.bias + (long long)f * a.n + o0 : nullptr;
    if (o0 + 4 <= a.n) {
        if (b) v += *reinterpret_cast<const f32x4_any *>(b);
        if constexpr (DT == BCONV_F32) {
            *reinterpret_cast<f32x4_any *>(y) = v;
        } else {
            typedef T Pair __attribute__((ext_vector_type(2)));
            const u32x2 p = {__builtin_bit_cast(uint32_t, (Pair){(T)v[0], (T)v[1]}), __builtin_bit_cast(uint32_t, (Pair){(T)v[2], (T)v[3]})};
            *reinterpret_cast<u32x2_any *>(y) = p;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (o0 + j < a.n) y[j] = (T)(b ? v[j] + b[j] : v[j]);
}

// One step's operand of 16 rows of x: codes of two instructions, their scales.
struct XStep {
    u32x4 c[2];
    uint32_t s;
};

// From elements: a lane's two blocks are 64 consecutive values of its row, so
// that quantising them asks no other lane.
template <int DT> __device__ __forceinline__ XStep quantised_step(const typename Elem<DT>::type *p, int left)
{
    XStep x;
    x.s = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        Eight<DT> e[4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e[j] = load_values<DT>(p + i * 32 + j * 8, left - i * 32 - j * 8);
            const uint32_t t = largest<DT>(e[j]);
            top = t > top ? t : top;
        }
        const uint32_t byte = scale_byte<DT>(top);
#pragma unroll
        for (int j = 0; j < 4; ++j) x.c[i][j] = to_codes<DT>(e[j], byte);
        x.s |= byte << (8 * i);
    }
    return x;
}

// Few rows of x for the weights.  A workgroup takes 16 RT outputs of one expert and its rows
// 16 at a time; its waves split the inputs step by step and add their sums in LDS, in
// a fixed order.
template <int DT, bool QUANTISED, int RT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void mx4_few_kernel(Mx4Args a)
{
    typedef typename Elem<DT>::type T;
    __shared__ f32x4 part[WAVES][RT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile0 = blockIdx.x * RT, row = lane & 15, lg = lane >> 4;
    const int f = a.offsets ? blockIdx.y : 0;
    Span span = expert_span(a, f);
    if (!a.offsets) {  // blockIdx.y counts 16 rows
        span.begin = blockIdx.y * 16;
        if (span.end > span.begin + 16) span.end = span.begin + 16;
    }
    if (f == a.experts) {  // rows of no expert
        for (int e = span.begin * RT * 4 + (int)threadIdx.x; e < span.end * RT * 4; e += WAVES * 64) {
            const int o0 = tile0 * 16 + e % (RT * 4) * 4;
            T *y = static_cast<T *>(a.y) + (long long)(e / (RT * 4)) * a.ldy + o0;
            for (int j = 0; j < 4; ++j)
                if (o0 + j < a.n) y[j] = (T)0.0f;
        }
        return;
    }
    for (int m0 = span.begin; m0 < span.end; m0 += 16) {
        const bool real = m0 + row < span.end;
        const long long xr = real ? input_row(a, m0 + row) : 0;
        f32x4 acc[RT];
        long long first[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            acc[r] = f32x4{0, 0, 0, 0};
            first[r] = ((long long)f * a.tiles + (tile0 + r < a.tiles ? tile0 + r : a.tiles - 1)) * a.steps;
        }
        // Lanes of columns past the last row load nothing: their operands stay 0,
        // and their results are not stored.
        XStep x = {{u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}}, 0};
        for (int c = wave; c < a.steps; c += WAVES) {
            u32x4 w[RT][2];
            uint32_t ws[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                w[r][0] = a.codes[(first[r] + c) * 128 + lane];
                w[r][1] = a.codes[(first[r] + c) * 128 + 64 + lane];
                ws[r] = a.scales[(first[r] + c) * 64 + lane];
            }
            if (real) {
                if constexpr (QUANTISED) {
                    const u32x4 *p = reinterpret_cast<const u32x4 *>(a.xc + (xr * a.steps + c) * (kStep / 2) + lg * 32);
                    x.c[0] = p[0];
                    x.c[1] = p[1];
                    x.s = *reinterpret_cast<const uint16_t *>(a.xs + (xr * a.steps + c) * (kStep / 32) + lg * 2);
                } else {
                    const int k0 = c * kStep + lg * 64;
                    x = quantised_step<DT>(static_cast<const T *>(a.x) + xr * a.ldx + k0, a.k - k0);
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r] = mfma_mx4<0>(w[r][0], ws[r], x.c[0], x.s, acc[r]);
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r] = mfma_mx4<1>(w[r][1], ws[r], x.c[1], x.s, acc[r]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) part[wave][r][lane] = acc[r];
        __syncthreads();
        for (int e = threadIdx.x; e < RT * 64; e += WAVES * 64) {
            const int l = e & 63, r = e >> 6;
            const int i = m0 + (l & 15), o0 = (tile0 + r) * 16 + (l >> 4) * 4;
            if (i >= span.end || o0 >= a.n) continue;
            f32x4 v = part[0][r][l];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += part[w][r][l];
            store_four<DT>(a, f, i, o0, v);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ many rows

// What the many-row kernel takes besides Mx4Args.
struct Mx4Many {
    float *sums;  // [splits][rows][padded_n], or nullptr for one split
    int row_blocks, out_blocks, splits;
    int padded_n;
};

// The row block `rb` of the launch: its expert and rows.  Experts' blocks follow each other,
// those of the rows of no expert come last; f is -1 behind them.
template <int R> __device__ __forceinline__ int find_rows(const Mx4Args &a, int rb, Span &span)
{
    if (!a.offsets) {
        span.begin = rb * R;
        span.end = a.rows - span.begin < R ? a.rows : span.begin + R;
        return 0;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;  // blocks of the experts before these 64
    for (int f0 = 0; f0 <= a.experts; f0 += 64) {
        const int f = f0 + lane;
        const Span s = f <= a.experts ? expert_span(a, f) : Span{0, 0};
        const int blocks = s.end > s.begin ? (s.end - s.begin + R - 1) / R : 0;
        int upto = blocks;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int u = __shfl_up(upto, d);
            if (lane >= d) upto += u;
        }
        const unsigned long long past = __ballot(before + upto > rb);
        if (past) {
            const int l = __builtin_ctzll(past);
            span.begin = __builtin_amdgcn_readlane(s.begin, l) + (rb - before - __builtin_amdgcn_readlane(upto - blocks, l)) * R;
            span.end = __builtin_amdgcn_readlane(s.end, l);
            if (span.end - span.begin > R) span.end = span.begin + R;
            return f0 + l;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return -1;
}

// A workgroup of WM x WN waves takes 16 WM MT rows of x and 16 WN NT outputs; a step
// of both (128 bytes a row) goes to LDS a step ahead, by loads that pass no registers.
template <int DT, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(WM * WN * 64, 2) void mx4_many_kernel(Mx4Args a, Mx4Many q)
{
    typedef typename Elem<DT>::type T;
    constexpr int WAVES = WM * WN, R = WM * MT * 16, OT = WN * NT;  // rows of x, output tiles
    constexpr int XL = R / 8 / WAVES, WL = OT * 2 / WAVES;         // 1 KiB loads a wave
    static_assert(XL * WAVES * 8 == R && WL * WAVES == OT * 2);
    struct Stage {
        u32x4 x[R * 8];    // [row][slot], block b of a step in slot b ^ (row >> 1 & 7)
        u32x4 w[OT * 128]; // [tile][instruction][lane]
    };
    __shared__ Stage stage[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, lg = lane >> 4;

    // Workgroups go to the XCDs in turn; each takes a run of neighbouring blocks.
    const int total = gridDim.x;
    int id = blockIdx.x;
    {
        const int xcd = id & 7, each = total >> 3, more = total & 7;
        id = xcd * each + (xcd < more ? xcd : more) + (id >> 3);
    }
    const int blocks = q.row_blocks * q.out_blocks;
    const int split = id / blocks;
    id -= split * blocks;
    constexpr int kGroup = 8;
    const int group = id / (kGroup * q.out_blocks), g0 = group * kGroup;
    const int high = q.row_blocks - g0 < kGroup ? q.row_blocks - g0 : kGroup;
    id -= group * kGroup * q.out_blocks;
    const int rb = g0 + id % high, ob = id / high;
    const int tile0 = ob * OT;

    Span span;
    const int f = find_rows<R>(a, rb, span);
    if (f < 0) return;
    if (f == a.experts) {  // rows of no expert
        for (int e = threadIdx.x; e < (span.end - span.begin) * OT * 16; e += WAVES * 64) {
            const int o = tile0 * 16 + e % (OT * 16);
            if (o < a.n) static_cast<T *>(a.y)[(long long)(span.begin + e / (OT * 16)) * a.ldy + o] = (T)0.0f;
        }
        return;
    }
    const int s_begin = (int)((long long)a.steps * split / q.splits), s_end = (int)((long long)a.steps * (split + 1) / q.splits);

    // where this lane's part of the loads comes from: rows past the last count as the last
    auto x_row = [&](int r) { return (uint32_t)input_row(a, min(span.begin + r, span.end - 1)); };
    const uint8_t *xp[XL];
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const int r = (j * WAVES + wave) * 8 + (lane >> 3);
        xp[j] = a.xc + (unsigned long long)x_row(r) * a.steps * 128 + ((lane & 7) ^ (r >> 1 & 7)) * 16;
    }
    const u32x4 *wp[WL];
#pragma unroll
    for (int j = 0; j < WL; ++j) {
        const int u = j * WAVES + wave, tile = min(tile0 + (u >> 1), a.tiles - 1);
        wp[j] = a.codes + (((long long)f * a.tiles + tile) * a.steps * 2 + (u & 1)) * 64 + lane;
    }
    const int my_x = wave / WN * MT * 16, my_tile = wave % WN * NT;
    uint32_t xs_at[MT];
    const uint16_t *ws_at[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xs_at[m] = x_row(my_x + m * 16 + row) * a.steps * 8 + lg * 2;
#pragma unroll
    for (int t = 0; t < NT; ++t)
        ws_at[t] = a.scales + ((long long)f * a.tiles + min(tile0 + my_tile + t, a.tiles - 1)) * a.steps * 64 + lane;

    typedef __attribute__((address_space(3))) void *Lds;
    uint32_t xs[MT], ws[NT], xn[MT], wn[NT];
    auto request = [&](int s) {
        Stage &st = stage[s & 1];
#pragma unroll
        for (int j = 0; j < XL; ++j)
            __builtin_amdgcn_global_load_lds((const void *)(xp[j] + (long long)s * 128), (Lds)(&st.x[(j * WAVES + wave) * 64]), 16, 0, 0);
#pragma unroll
        for (int j = 0; j < WL; ++j)
            __builtin_amdgcn_global_load_lds((const void *)(wp[j] + (long long)s * 128), (Lds)(&st.w[(j * WAVES + wave) * 64]), 16, 0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) xn[m] = *reinterpret_cast<const uint16_t *>(a.xs + (size_t)s * 8 + xs_at[m]);
#pragma unroll
        for (int t = 0; t < NT; ++t) wn[t] = ws_at[t][s * 64];
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0, 0, 0, 0};
    if (s_begin < s_end) request(s_begin);
    for (int s = s_begin; s < s_end; ++s) {
        __builtin_amdgcn_s_waitcnt(0 | (0x7 << 4) | (0xf << 8));  // vmcnt(0): this step's operands are here
        __syncthreads();                                          // in every wave, and the other stage is read
#pragma unroll
        for (int m = 0; m < MT; ++m) xs[m] = xn[m];
#pragma unroll
        for (int t = 0; t < NT; ++t) ws[t] = wn[t];
        if (s + 1 < s_end) request(s + 1);
        const Stage &st = stage[s & 1];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u32x4 w[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) w[t] = st.w[((my_tile + t) * 2 + i) * 64 + lane];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = my_x + m * 16 + row;
                const u32x4 x = st.x[r * 8 + ((2 * lg + i) ^ (r >> 1 & 7))];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    acc[m][t] = i ? mfma_mx4<1>(w[t], ws[t], x, xs[m], acc[m][t]) : mfma_mx4<0>(w[t], ws[t], x, xs[m], acc[m][t]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = span.begin + my_x + m * 16 + row;
        if (i >= span.end) continue;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int o0 = (tile0 + my_tile + t) * 16 + lg * 4;
            if (q.splits > 1)
                *reinterpret_cast<f32x4 *>(q.sums + ((long long)split * a.rows + i) * q.padded_n + o0) = acc[m][t];
            else if (o0 < a.n) store_four<DT>(a, f, i, o0, acc[m][t]);
        }
    }
}

// Adds the splits' sums in order.
template <int DT> __global__ __launch_bounds__(256) void mx4_join_kernel(Mx4Args a, Mx4Many q)
{
    const int per = (a.n + 3) / 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long long)per * a.rows) return;
    const int i = (int)(id / per), o0 = (int)(id % per) * 4;
    const float *p = q.sums + (long long)i * q.padded_n + o0;
    const long long step = (long long)a.rows * q.padded_n;
    f32x4 v = *reinterpret_cast<const f32x4 *>(p);
    for (int s = 1; s < q.splits; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * step);
    store_four<DT>(a, 0, i, o0, v);
}

// ------------------------------------------------------------------ dispatch

struct Mx4Plan {
    bool quantise;  // x is quantised by a launch of its own
    int shape;      // 0: few rows; rows of x of the many-row kernel's workgroup
    Mx4Many q;
    size_t scales_offset, sums_offset, bytes;
};

Mx4Plan plan_mx4(const Mx4Args &a, bool given, int cus)
{
    Mx4Plan p{};
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const int mean = a.rows / a.experts;
    p.shape = mean > 512 ? 256 : mean > 16 ? 128 : 0;
    p.quantise = !given && (a.rows > 4 || p.shape);
    if (p.quantise) {
        p.scales_offset = (size_t)a.x_rows * a.steps * (kStep / 2);
        p.bytes = p.sums_offset = up(p.scales_offset + (size_t)a.x_rows * a.steps * (kStep / 32));
    }
    if (p.shape) {
        const int out_tiles = p.shape / 16;
        p.q.row_blocks = (a.rows + p.shape - 1) / p.shape + (a.offsets ? a.experts : 0);
        p.q.out_blocks = (a.tiles + out_tiles - 1) / out_tiles;
        p.q.padded_n = p.q.out_blocks * p.shape;
        p.q.splits = 1;
        if (!a.offsets) {
            const long long blocks = (long long)p.q.row_blocks * p.q.out_blocks;
            long long splits = (2LL * cus) / blocks;
            if (splits > 8) splits = 8;
            if (splits > a.steps / 4) splits = a.steps / 4;
            p.q.splits = splits < 1 ? 1 : (int)splits;
        }
        if (p.q.splits > 1) p.bytes = p.sums_offset + (size_t)p.q.splits * a.rows * p.q.padded_n * 4;
    }
    return p;
}

template <int DT> hipError_t run_mx4(const Mx4Args &a, const Mx4Plan &p, hipStream_t s)
{
    if (p.shape) {
        const dim3 grid((unsigned)((long long)p.q.row_blocks * p.q.out_blocks * p.q.splits));
        if (p.shape == 256) hipLaunchKernelGGL((mx4_many_kernel<DT, 2, 4, 8, 4>), grid, dim3(512), 0, s, a, p.q);
        else hipLaunchKernelGGL((mx4_many_kernel<DT, 2, 2, 4, 4>), grid, dim3(256), 0, s, a, p.q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.q.splits == 1) return e;
        const long long outs = (long long)((a.n + 3) / 4) * a.rows;
        hipLaunchKernelGGL((mx4_join_kernel<DT>), dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, s, a, p.q);
        return hipGetLastError();
    }
    const dim3 grid((a.tiles + 1) / 2, a.offsets ? a.experts + 1 : (a.rows + 15) / 16);
    if (a.x) hipLaunchKernelGGL((mx4_few_kernel<DT, false, 2, 8>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((mx4_few_kernel<DT, true, 2, 8>), grid, dim3(512), 0, s, a);
    return hipGetLastError();
}

}  // namespace bconv

struct bconv_mx4_linear {
    bconv_mx4_linear_desc_t desc;
    int device, cus;
    int tiles, steps;
    uint32_t *d_codes;
    uint8_t *d_scales;
    float *d_bias;
};

namespace {

using bconv::DeviceGuard;
using bconv::fail;
using bconv::hip_fail;
using bconv::ranges_overlap;

constexpr int32_t kMaxFeatures = 1 << 20;

bconv_status_t check_desc(const bconv_mx4_linear_desc_t *d)
{
    if (!d) return fail(BCONV_ERR_INVALID_ARGUMENT, "desc is NULL");
    if (d->experts < 1 || d->experts > 1024) return fail(BCONV_ERR_INVALID_ARGUMENT, "experts must be in [1, 1024]");
    if (d->in_features < 1 || d->in_features > kMaxFeatures || d->out_features < 1 || d->out_features > kMaxFeatures)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "in_features/out_features must be in [1, %d]", kMaxFeatures);
    if ((long long)d->in_features * d->out_features > (1LL << 38) / d->experts)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "experts*in_features*out_features exceeds 2^38");
    return BCONV_OK;
}

void release(bconv_mx4_linear *h)
{
    void *ptrs[] = {h->d_codes, h->d_scales, h->d_bias};
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

// What sizes alone decide of a call; workspace_size and forward share it.
bconv_status_t check_sizes(bconv_mx4_linear_t h, const bconv_mx4_rows_t *args)
{
    if (!h || !args) return fail(BCONV_ERR_INVALID_ARGUMENT, "handle or args is NULL");
    if (args->rows < 0 || args->x_rows < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows and x_rows must be >= 0");
    if (!dtype_bytes(args->dtype)) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", args->dtype);
    if (args->choices < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "choices must be >= 0");
    if (args->choices == 0 ? args->x_rows != args->rows : (long long)args->x_rows * args->choices != args->rows)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "%d rows do not follow from %d input rows and %d choices", args->rows,
                    args->x_rows, args->choices);
    return BCONV_OK;
}

bconv::Mx4Args kernel_args(bconv_mx4_linear_t h, const bconv_mx4_rows_t *args)
{
    bconv::Mx4Args a{};
    a.codes = reinterpret_cast<const bconv::u32x4 *>(h->d_codes);
    a.scales = reinterpret_cast<const uint16_t *>(h->d_scales);
    a.bias = h->d_bias;
    a.x = args->x;
    a.xc = args->codes;
    a.xs = args->scales;
    a.y = args->y;
    a.offsets = args->offsets;
    a.order = args->order;
    a.ldx = args->ldx;
    a.ldy = args->ldy;
    a.rows = args->rows;
    a.x_rows = args->x_rows;
    a.choices = args->choices;
    a.n = h->desc.out_features;
    a.k = h->desc.in_features;
    a.tiles = h->tiles;
    a.steps = h->steps;
    a.experts = h->desc.experts;
    return a;
}

}  // namespace

extern "C" {

bconv_status_t bconv_mx4_linear_create(const bconv_mx4_linear_desc_t *desc, void *stream, const uint8_t *codes,
                                       const uint8_t *scales, const float *bias, bconv_mx4_linear_t *out)
{
    if (!out) return fail(BCONV_ERR_INVALID_ARGUMENT, "out is NULL");
    *out = nullptr;
    bconv_status_t st = check_desc(desc);
    if (st != BCONV_OK) return st;
    if (!codes || !scales) return fail(BCONV_ERR_INVALID_ARGUMENT, "codes or scales is NULL");
    if ((uintptr_t)bias % 4) return fail(BCONV_ERR_INVALID_ARGUMENT, "bias not aligned to an element");
    const int n = desc->out_features, k = desc->in_features;
    bconv_mx4_linear *h = new (std::nothrow) bconv_mx4_linear();
    if (!h) return fail(BCONV_ERR_ALLOC, "host allocation failed");
    h->desc = *desc;
    h->tiles = (n + 15) / 16;
    h->steps = (int)(bconv::mx4_padded(k) / bconv::kStep);
    hipError_t e = hipGetDevice(&h->device);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, h->device);
    if (e != hipSuccess) {
        release(h);
        return hip_fail(e, "hipGetDevice");
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const long long cells = (long long)desc->experts * h->tiles * h->steps;
    const size_t nb = (size_t)desc->experts * n;
    if ((st = device_alloc(&h->d_codes, (size_t)cells * 512)) == BCONV_OK &&
        (st = device_alloc(&h->d_scales, (size_t)cells * 128)) == BCONV_OK &&
        (!bias || (st = device_alloc(&h->d_bias, nb)) == BCONV_OK)) {
        e = bconv::launch_slices(cells * 2, [&](long long first, unsigned groups) {
            hipLaunchKernelGGL(bconv::mx4_prepack_kernel, dim3(groups), dim3(256), 0, s, codes, h->d_codes, n, k, h->tiles,
                               h->steps, first * 256, cells * 512);
        });
        if (e == hipSuccess)
            e = bconv::launch_slices((cells + 1) / 2, [&](long long first, unsigned groups) {
                hipLaunchKernelGGL(bconv::mx4_prepack_scales_kernel, dim3(groups), dim3(256), 0, s, scales, h->d_scales, n, k,
                                   h->tiles, h->steps, first * 256, cells * 128);
            });
        if (e == hipSuccess && bias) e = hipMemcpyAsync(h->d_bias, bias, nb * sizeof(float), hipMemcpyDeviceToDevice, s);
        const hipError_t done = hipStreamSynchronize(s);  // also after an error: a launch may still read the caller's buffers
        if (e == hipSuccess) e = done;
        if (e != hipSuccess) st = hip_fail(e, "weight layout");
    }
    if (st != BCONV_OK) {
        release(h);
        return st;
    }
    *out = h;
    return BCONV_OK;
}

bconv_status_t bconv_mx4_linear_workspace_size(bconv_mx4_linear_t h, const bconv_mx4_rows_t *args, size_t *bytes)
{
    const bconv_status_t st = check_sizes(h, args);
    if (st != BCONV_OK) return st;
    if (!bytes) return fail(BCONV_ERR_INVALID_ARGUMENT, "bytes is NULL");
    *bytes = args->rows ? bconv::plan_mx4(kernel_args(h, args), !args->x, h->cus).bytes : 0;
    return BCONV_OK;
}

bconv_status_t bconv_mx4_linear_forward(bconv_mx4_linear_t h, void *stream, const bconv_mx4_rows_t *args, void *workspace,
                                        size_t workspace_bytes)
{
    bconv_status_t st = check_sizes(h, args);
    if (st != BCONV_OK) return st;
    if (args->rows == 0) return BCONV_OK;
    const int es = dtype_bytes(args->dtype), n = h->desc.out_features, k = h->desc.in_features;
    if (!args->y || (!args->x && (!args->codes || !args->scales)))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "y and x (or codes and scales) must not be NULL");
    if (args->x && (args->codes || args->scales)) return fail(BCONV_ERR_INVALID_ARGUMENT, "x and codes are both given");
    if (args->ldy < n || args->ldy > (1LL << 40)) return fail(BCONV_ERR_INVALID_ARGUMENT, "ldy must be in [out_features, 2^40]");
    if (args->x && (args->ldx < k || args->ldx > (1LL << 40)))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "ldx must be in [in_features, 2^40]");
    if (((uintptr_t)args->x | (uintptr_t)args->y) % es) return fail(BCONV_ERR_INVALID_ARGUMENT, "x/y not aligned to an element");
    if ((uintptr_t)args->codes % 16 || (uintptr_t)args->scales % 8)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned, scales 8-byte");
    if (!args->offsets && h->desc.experts > 1) return fail(BCONV_ERR_INVALID_ARGUMENT, "offsets is NULL, the layer has experts");
    if ((args->choices > 0) != (args->order != nullptr))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "order must be given with choices, and only then");
    if (((uintptr_t)args->offsets | (uintptr_t)args->order) % 4)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "offsets/order not aligned to an element");
    bconv::Mx4Args a = kernel_args(h, args);
    bconv::Mx4Plan p = bconv::plan_mx4(a, !args->x, h->cus);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes))
        return fail(BCONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.bytes, workspace ? workspace_bytes : (size_t)0);
    if (p.bytes > 0 && (uintptr_t)workspace % 16) return fail(BCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    const size_t xc = (size_t)args->x_rows * h->steps * (bconv::kStep / 2), xs = xc / 16;
    const struct { const void *p; size_t n; } in[] = {
        {args->x, args->x ? ((size_t)(args->x_rows - 1) * args->ldx + k) * es : 0}, {args->codes, args->codes ? xc : 0},
        {args->scales, args->scales ? xs : 0}, {args->offsets, args->offsets ? ((size_t)h->desc.experts + 1) * 4 : 0},
        {args->order, args->order ? (size_t)args->rows * 4 : 0}},
        out[] = {{args->y, ((size_t)(args->rows - 1) * args->ldy + n) * es}, {workspace, p.bytes}};
    for (const auto &o : out)
        for (const auto &i : in)
            if (o.n && i.n && ranges_overlap(o.p, o.n, i.p, i.n))
                return fail(BCONV_ERR_INVALID_ARGUMENT, "y or the workspace overlaps x, codes, scales, offsets or order");
    if (p.bytes && ranges_overlap(out[0].p, out[0].n, workspace, p.bytes))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "y and the workspace overlap");

    DeviceGuard guard(h->device);
    if (guard.err != hipSuccess) return hip_fail(guard.err, "hipSetDevice");
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = hipSuccess;
    if (p.quantise) {
        uint8_t *codes = static_cast<uint8_t *>(workspace);
        e = bconv::mx4_quantize_rows(s, a.x_rows, k, args->dtype, a.x, a.ldx, codes, codes + p.scales_offset, nullptr);
        if (e != hipSuccess) return hip_fail(e, "mx4 quantisation kernel");
        a.x = nullptr;
        a.xc = codes;
        a.xs = codes + p.scales_offset;
    }
    p.q.sums = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.sums_offset);
    switch (args->dtype) {
    case BCONV_F32: e = bconv::run_mx4<BCONV_F32>(a, p, s); break;
    case BCONV_F16: e = bconv::run_mx4<BCONV_F16>(a, p, s); break;
    default: e = bconv::run_mx4<BCONV_BF16>(a, p, s); break;
    }
    if (e != hipSuccess) return hip_fail(e, "mx4 linear kernel");
    return BCONV_OK;
}

bconv_status_t bconv_mx4_linear_destroy(bconv_mx4_linear_t h)
{
    if (!h) return BCONV_OK;
    DeviceGuard guard(h->device);
    release(h);
    return BCONV_OK;
}

}  // extern "C"
