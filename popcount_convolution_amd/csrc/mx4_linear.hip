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
#include <type_traits>

#include "host.h"
#include "mx4.h"

namespace bconv {

// A layer's weights: [experts][tiles][steps][2][64 lanes][16 bytes], scales
// [experts][tiles][steps][16 outputs][8 blocks].
struct Mx4Args {
    const u32x4 *codes;
    const uint8_t *scales;
    const float *bias;       // [experts][n] or nullptr
    const void *x;           // elements, or nullptr
    const uint8_t *xc, *xs;  // quantised rows; the scales of a row's step are 8 bytes,
    long long xs_row, xs_step;  // this far from the next row's and step's
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
    const int block = (int)(id & 7), r = (int)(id >> 3) & 15;
    id >>= 7;
    const int step = (int)(id % steps);
    id /= steps;
    const int tile = (int)(id % tiles);
    const long long f = id / tiles;
    const int o = tile * 16 + r, b = step * (kStep / 32) + block, blocks = (k + 31) / 32;
    *to = o < n && b < blocks ? user[(f * n + o) * blocks + b] : 0;
}

__device__ __forceinline__ Span expert_span(const Mx4Args &a, int f)
{
    if (!a.offsets) return {0, a.rows};
    return expert_rows(a.offsets, a.experts, a.rows, f);
}

// Input row of result row i (i < rows): what pair_of() loads, then input_row().
__device__ __forceinline__ int pair_of(const Mx4Args &a, int i) { return a.choices == 0 ? i : a.order[i]; }

__device__ __forceinline__ int input_row(const Mx4Args &a, int pair)
{
    if (a.choices == 0) return pair;
    const int r = pair < 0 ? 0 : pair / a.choices;
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

// Few rows of x for the weights.  A workgroup takes 16 RT outputs of one expert and
// its rows 16 CT at a time; its waves split the inputs step by step and add their
// sums in LDS, in a fixed order.  The weights go from global memory to the matrix
// cores without passing LDS, as in memory.
//
// Bound by the weights' bytes: 1 x 25088 -> 4096, 54.6 MB, 9.4 to 9.5 us (5.7 to 5.8 TB/s;
// a large read reaches 5.8), after 2.9 us that quantise the row; 13 x 5000 -> 11003 fp32, 30 MB, 6.2 to 7.2 us
// (4.2 to 4.9 TB/s: a wave has one step's loads in flight) after 3.8; 32 tokens' 4 of 64 experts of 2048 -> 2816,
// of which they choose 44, 135 MB, 20 to 22 us (6.1 to 6.8 TB/s, some of it in the memory-side cache) after 2.5 to 4.
// 512 -> 512: 3.1 us, the launch and a chain of loads.
template <int DT, bool QUANTISED, int RT, int CT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void mx4_few_kernel(Mx4Args a)
{
    typedef typename Elem<DT>::type T;
    __shared__ f32x4 part[WAVES][RT * CT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile0 = blockIdx.x * RT, row = lane & 15, lg = lane >> 4;
    const int f = a.offsets ? blockIdx.y : 0;
    Span span = expert_span(a, f);
    if (!a.offsets) {  // blockIdx.y counts blocks of rows
        span.begin = blockIdx.y * (16 * CT);
        if (span.end > span.begin + 16 * CT) span.end = span.begin + 16 * CT;
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
    long long first[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) first[r] = ((long long)f * a.tiles + (tile0 + r < a.tiles ? tile0 + r : a.tiles - 1)) * a.steps;
    for (int m0 = span.begin; m0 < span.end; m0 += 16 * CT) {
        f32x4 acc[RT][CT];
        // Lanes of columns past the last row load nothing: their operands stay 0,
        // and their results are not stored.
        XStep x[CT];
        long long xr[CT];
        bool real[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            real[t] = m0 + t * 16 + row < span.end;
            xr[t] = real[t] ? input_row(a, pair_of(a, m0 + t * 16 + row)) : 0;
            x[t] = {{u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}}, 0};
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r][t] = f32x4{0, 0, 0, 0};
        }
        for (int c = wave; c < a.steps; c += WAVES) {
            u32x4 w[RT][2];
            uint32_t ws[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                w[r][0] = a.codes[(first[r] + c) * 128 + lane];
                w[r][1] = a.codes[(first[r] + c) * 128 + 64 + lane];
                ws[r] = *reinterpret_cast<const uint16_t *>(a.scales + (first[r] + c) * 128 + row * 8 + lg * 2);
            }
#pragma unroll
            for (int t = 0; t < CT; ++t)
                if (real[t]) {
                    if constexpr (QUANTISED) {
                        const u32x4 *p = reinterpret_cast<const u32x4 *>(a.xc + (xr[t] * a.steps + c) * (kStep / 2) + lg * 32);
                        x[t].c[0] = p[0];
                        x[t].c[1] = p[1];
                        x[t].s = *reinterpret_cast<const uint16_t *>(a.xs + xr[t] * a.xs_row + c * a.xs_step + lg * 2);
                    } else {
                        const int k0 = c * kStep + lg * 64;
                        x[t] = quantised_step<DT>(static_cast<const T *>(a.x) + xr[t] * a.ldx + k0, a.k - k0);
                    }
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < CT; ++t)
                        acc[r][t] = i ? mfma_mx4<1>(w[r][1], ws[r], x[t].c[1], x[t].s, acc[r][t])
                                      : mfma_mx4<0>(w[r][0], ws[r], x[t].c[0], x[t].s, acc[r][t]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < CT; ++t) part[wave][r * CT + t][lane] = acc[r][t];
        __syncthreads();
        for (int e = threadIdx.x; e < RT * CT * 64; e += WAVES * 64) {
            const int l = e & 63, u = e >> 6;
            const int i = m0 + u % CT * 16 + (l & 15), o0 = (tile0 + u / CT) * 16 + (l >> 4) * 4;
            if (i >= span.end || o0 >= a.n) continue;
            f32x4 v = part[0][u][l];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += part[w][u][l];
            store_four<DT>(a, f, i, o0, v);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ many rows
//
// Four waves lie along the outputs and share 128 rows of x: x goes through LDS,
// where every wave reads all of it, while a wave's weights are its own and go
// from global memory to its registers in the order that they were laid out in.
// x's stages are requested three steps ahead, by loads that pass no registers,
// weights one step (three, in the narrow shape); the loads, 10 to 15 a step, lie
// between the matrix instructions one by one, so that neither waits for the
// other's issue.  32x32x64 instructions: with scales and random codes, one wave a
// SIMD reaches 6.4 PFLOP/s with them and 4.2 with 16x16x128 (9.1 and 5.1 on zeros:
// the clock falls with the bits that toggle).
//
// Bound by power for large products: 8192 x 8192 -> 8192 bf16, 231 to 280 us (3.9 to
// 4.8 PFLOP/s, 3.3 to 4 times a large bf16 library product), matrix cores busy 71 to 74%
// of the cycles at 1.3 to 1.5 GHz (an earlier form took as many cycles on zeros, at
// 2.3 GHz instead of 1.7).  On the way there: both operands in LDS with 16x16x128
// instructions 435 to 460 us, with 32x32x64 330 to 370, weights in registers 320,
// results as whole lines 285, a ring of register sets and exact waits 250.
// For experts by the weights' and results' bytes: 16396 rows of 64 experts, 2048 ->
// 2816, 327 MB moved, 67 to 77 us (4.2 to 4.9 TB/s, a copy's rate).  256 x 25088 -> 4096, 19 to 21 us, by the
// latency of the weights, three steps ahead in 256 workgroups of one wave a SIMD.

// What the many-row kernel takes besides Mx4Args.
struct Mx4Many {
    float *sums;  // [splits][rows][padded_n], or nullptr for one split
    const RowBlock *row_list;  // with experts: what make_row_blocks() makes
    int row_blocks, out_blocks, splits;
    int padded_n;
    int first;    // the launch's first workgroup
};

// The list of row blocks, where no other launch makes it.
__global__ __launch_bounds__(kListThreads) void mx4_blocks_kernel(RowBlocks b) { make_row_blocks(b); }

template <typename E> struct Values {  // of 16 bytes
    E v[16 / sizeof(E)];
};

// s_waitcnt: at most `n` vector loads outstanding, no LDS read.
constexpr int vm_wait(int n) { return (n & 15) | (n >> 4 << 14) | (0x7 << 4) | (0x0 << 8); }

// Bytes of every buffer, so that an offset from there on reads no memory and gives
// 0.  Quantised rows may fill it: with a byte less, the last codes of the last row read as 0.
constexpr uint32_t kNone = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t whole_buffer(const void *p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, kNone, 0x00020000);
}

// LDS of the many-row kernel.
template <int MT> struct ManyStage {
    u32x4 x[MT * 32 * 8];      // [row][slot], block b of a step in slot b ^ (row >> 1 & 7)
    uint32_t xs[MT * 32 * 2];  // [row][half]
};

constexpr int kStages = 4, kManyRows = 128;

union ManyLds {
    ManyStage<kManyRows / 32> stage[kStages];
    char out[4096 * 4];  // results on their way out, a wave's after the other's
};

// Results of up to 32 MT rows of expert f, 128 NT outputs from tile0 on.
template <int DT, int MT, int NT, int WD>
__device__ __forceinline__ void many_rows(const Mx4Args &a, const Mx4Many &q, ManyLds &lds, int f, Span span, int tile0, int split)
{
    typedef typename Elem<DT>::type T;
    constexpr int WAVES = 4, STAGES = kStages, R = MT * 32;
    constexpr int XL = R / 8 / WAVES, XV = XL + 1, WV = 5 * NT;  // loads of a step: x and its scales, weights and theirs
    static_assert(R <= kManyRows);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 31, half = lane >> 5;
    const int s_begin = __builtin_amdgcn_readfirstlane((int)((long long)a.steps * split / q.splits));
    const int s_end = __builtin_amdgcn_readfirstlane((int)((long long)a.steps * (split + 1) / q.splits));

    // Where this lane's part of the loads comes from: rows and tiles past the last
    // count as the last.  Offsets stay below kNone.
    const long long x_base = a.choices ? 0 : span.begin;
    const int my_scales = wave % MT * 32;  // with few rows, several waves load the same
    int pair[XL + 1];
#pragma unroll
    for (int j = 0; j <= XL; ++j) {
        const int r = j < XL ? (j * WAVES + wave) * 8 + (lane >> 3) : my_scales + (lane >> 1);
        pair[j] = pair_of(a, min(span.begin + r, span.end - 1));
    }
    uint32_t xo[XL], xso, wo[NT], wso[NT];
    const int my_tile = tile0 + wave * NT * 2;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const uint32_t tile = min(my_tile + t * 2 + (row >> 4), a.tiles - 1) - tile0;
        wo[t] = tile * a.steps * 2048 + half * 512 + (row & 15) * 16;
        wso[t] = tile * a.steps * 128 + (row & 15) * 8 + half * 4;
    }
    const long long first_tile = (long long)f * a.tiles + tile0;
    const __amdgpu_buffer_rsrc_t rxc = whole_buffer(a.xc + x_base * a.steps * 128), rxs = whole_buffer(a.xs + x_base * a.xs_row);
    const __amdgpu_buffer_rsrc_t rwc = whole_buffer(a.codes + first_tile * a.steps * 128);
    const __amdgpu_buffer_rsrc_t rws = whole_buffer(a.scales + first_tile * a.steps * 128);
    const int xs_step = __builtin_amdgcn_readfirstlane((int)a.xs_step);

    typedef __attribute__((address_space(3))) void *Lds;
    auto request_x = [&](int s, int slot, int l) {  // one of XV
        ManyStage<kManyRows / 32> &st = lds.stage[slot];
        const uint32_t none = s < s_end ? 0 : kNone;
        if (l == 0)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (Lds)(&st.xs[my_scales * 2]), 4, (int)(xso | none), s * xs_step, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rxc, (Lds)(&st.x[((l - 1) * WAVES + wave) * 64]), 16, (int)(xo[l - 1] | none), s * 128, 0, 0);
    };
    u32x4 w[WD + 1][4][NT];
    uint32_t ws[WD + 1][NT];
    auto request_w = [&](int s, int set, int l) {  // one of WV
        const uint32_t none = s < s_end ? 0 : kNone;
        if (l < NT) ws[set][l] = __builtin_amdgcn_raw_buffer_load_b32(rws, (int)(wso[l] | none), s * 128, 0);
        else {
            const int i = (l - NT) / NT, t = (l - NT) % NT;
            w[set][i][t] = __builtin_amdgcn_raw_buffer_load_b128(rwc, (int)(wo[t] | none), s * 2048 + (i & 1) * 1024 + (i >> 1) * 256, 0);
        }
    };
    f32x16 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][t][i] = 0.0f;
    u32x4 x[2][MT];
    uint32_t xs[2][MT];
    auto fetch = [&](int slot, int i, int m) {
        const int r = m * 32 + row;
        x[i & 1][m] = lds.stage[slot].x[r * 8 + ((4 * half + i) ^ (r >> 1 & 7))];
    };
    auto fetch_scale = [&](int slot, int m) { xs[slot & 1][m] = lds.stage[slot].xs[(m * 32 + row) * 2 + half]; };
    // Step s, whose x is in stage `at` = (s - s_begin) % 4.  LEFT: the steps that
    // may still follow, as far as that is known: x of s + 3 and weights of s + WD are
    // requested where there can be such a step.  What the wait counts has to be
    // issued as written: a load whose result no step uses would be dropped.
    constexpr int V = WV + XV, P = MT * NT;  // loads of a whole step, instructions a phase
    auto step = [&](int s, auto AT, auto LEFT) {
        constexpr int at = decltype(AT)::value, next = (at + 1) & 3, left = decltype(LEFT)::value;
        constexpr int loads = (left >= WD ? WV : 0) + (left >= STAGES - 1 ? XV : 0);
        constexpr int before = at > 0 && left < STAGES - 1 ? (left + 1 >= WD ? WV : 0) : V;  // loads of the step before
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i == 3 && left > 0) {
                // x of the next step is here: all loads but those after it are done
                __builtin_amdgcn_s_waitcnt(vm_wait(before + loads));
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int m = p / NT, t = p % NT;
                if (t == 0) {
                    if (i < 3) fetch(at, i + 1, m);
                    else if (left > 0) {
                        fetch_scale(next, m);
                        fetch(next, 0, m);
                    }
                }
                if (i < 3) {
                    // the loads spread over three phases
#pragma unroll
                    for (int l = 0; l < V; ++l)
                        if (l * 3 * P / V == i * P + p) {
                            if (l < WV) {
                                if constexpr (left >= WD) request_w(s + WD, (at + WD) % (WD + 1), l);
                            } else if constexpr (left >= STAGES - 1) {
                                request_x(s + STAGES - 1, (at + STAGES - 1) & 3, l - WV);
                            }
                        }
                }
                acc[m][t] = mfma_mx4_32(i, w[at % (WD + 1)][i][t], ws[at % (WD + 1)][t], x[i & 1][m], xs[at & 1][m], acc[m][t]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    static_assert(4 % (WD + 1) == 0 && WD < STAGES && 2 * V < 64);
    // the first weights are on their way while the pairs arrive that say which rows of x
#pragma unroll
    for (int d = 0; d < WD; ++d)
#pragma unroll
        for (int l = 0; l < WV; ++l) request_w(s_begin + d, d, l);
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const int r = (j * WAVES + wave) * 8 + (lane >> 3);
        xo[j] = (uint32_t)(input_row(a, pair[j]) - x_base) * a.steps * 128 + ((lane & 7) ^ (r >> 1 & 7)) * 16;
    }
    xso = (uint32_t)((input_row(a, pair[XL]) - x_base) * a.xs_row + (lane & 1) * 4);
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d)
#pragma unroll
        for (int l = 0; l < XV; ++l) request_x(s_begin + d, d, l);
    __builtin_amdgcn_s_waitcnt(vm_wait(0));  // x of three steps is here
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        fetch_scale(0, m);
        fetch(0, 0, m);
    }
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;
    typedef std::integral_constant<int, 2> I2;
    typedef std::integral_constant<int, 3> I3;
    int s = s_begin;
    for (; s + 4 <= s_end; s += 4) {  // up to three more may follow the last
        step(s, I0(), I3());
        step(s + 1, I1(), I3());
        step(s + 2, I2(), I3());
        step(s + 3, I3(), I3());
    }
    if (s < s_end) {
        step(s, I0(), I2());
        if (s + 1 < s_end) {
            step(s + 1, I1(), I1());
            if (s + 2 < s_end) step(s + 2, I2(), I0());
        }
    }
    __builtin_amdgcn_s_waitcnt(vm_wait(0));  // nothing is on its way to LDS any more,
    __builtin_amdgcn_s_barrier();            // of any wave
    // Results through LDS, 32 rows of up to 128 bytes a wave at a time, so that they leave as whole lines.
    const int y0 = my_tile * 16;  // the wave's first output
    char *out = lds.out + wave * 4096;
    auto emit = [&](auto TYPE, auto AWAY, auto &result, char *to, long long ld, int n) {
        typedef decltype(TYPE) E;
        constexpr int TT = sizeof(E) == 2 ? NT : 1, CH = TT * 2 * (int)sizeof(E);  // blocks of 32 outputs, 16-byte pieces a row
        constexpr int PER = 16 / (int)sizeof(E);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t0 = 0; t0 < NT; t0 += TT) {
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {  // results 4 v + j are outputs 8 v + 4 half + j of the 32
                        const f32x4 r = result(m, t0 + t, v);
                        typedef E E4 __attribute__((ext_vector_type(4)));
                        const E4 e = {(E)r[0], (E)r[1], (E)r[2], (E)r[3]};
                        const int at = (t * 32 + v * 8 + half * 4) * (int)sizeof(E);
                        *reinterpret_cast<E4 *>(out + row * (CH * 16) + (((at >> 4) ^ row) & (CH - 1)) * 16 + (at & 15)) = e;
                    }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int k = 0; k < CH / 2; ++k) {
                    const int r = k * (64 / CH) + lane / CH, c = lane % CH;
                    const u32x4 e = *reinterpret_cast<const u32x4 *>(out + r * (CH * 16) + ((c ^ r) & (CH - 1)) * 16);
                    const int i = m * 32 + r, o = y0 + t0 * 32 + c * PER;
                    if (span.begin + i >= span.end) continue;
                    char *p = to + ((long long)i * ld + o) * (int)sizeof(E);
                    if (o + PER <= n) {
                        u32x4_any *to16 = reinterpret_cast<u32x4_any *>(p);
                        if constexpr (decltype(AWAY)::value) __builtin_nontemporal_store(e, to16);
                        else *to16 = e;
                    }
                    else {
#pragma unroll
                        for (int x = 0; x < PER; ++x)
                            if (o + x < n) reinterpret_cast<E *>(p)[x] = __builtin_bit_cast(Values<E>, e).v[x];
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
    };
    if (q.splits > 1) {
        auto plain = [&](int m, int t, int v) {
            return f32x4{acc[m][t][4 * v], acc[m][t][4 * v + 1], acc[m][t][4 * v + 2], acc[m][t][4 * v + 3]};
        };
        emit(0.0f, std::false_type(), plain,
             reinterpret_cast<char *>(q.sums + ((long long)split * a.rows + span.begin) * q.padded_n), q.padded_n, q.padded_n);
    } else {
        f32x4 bias[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int o = y0 + t * 32 + v * 8 + half * 4;
                bias[t][v] = f32x4{0, 0, 0, 0};
                if (!a.bias || o >= a.n) continue;
                const float *b = a.bias + (long long)f * a.n + o;
                if (o + 4 <= a.n) bias[t][v] = *reinterpret_cast<const f32x4_any *>(b);
                else
                    for (int j = 0; j < a.n - o; ++j) bias[t][v][j] = b[j];
            }
        auto biased = [&](int m, int t, int v) {
            return f32x4{acc[m][t][4 * v], acc[m][t][4 * v + 1], acc[m][t][4 * v + 2], acc[m][t][4 * v + 3]} + bias[t][v];
        };
        // past the caches, whose room the weights and x of other workgroups need (quantise and product of 16396 rows, 64
        // experts of 2048 -> 2816: 86 us, 73 so; 4096 rows, 16 of 1024 -> 1408: 16.7, 15.6), at any size: with a kernel
        // that reads the results next, 128 and 131; 28.1 and 24.3; 1024 rows, 8 of 2048 -> 2816 19.2 and 18.9; one layer, 512 x
        // 1024 -> 4096 14.4 and 14.7, 2048 x 4096 -> 4096 38.2 and 37.7, 8192 x 8192 -> 8192 350 and 328
        emit(T(), std::true_type(), biased, reinterpret_cast<char *>(static_cast<T *>(a.y) + (long long)span.begin * a.ldy), a.ldy, a.n);
    }
}

template <int DT, int NT, int WD>
__global__ __launch_bounds__(256, 2) void mx4_many_kernel(Mx4Args a, Mx4Many q)
{
    typedef typename Elem<DT>::type T;
    constexpr int OT = NT * 8;  // tiles of 16 outputs
    __shared__ ManyLds lds;
    // Workgroups go to the XCDs in turn; each takes a run of neighbouring blocks.
    const int row_blocks = q.row_list ? q.row_list[0].f : q.row_blocks;
    const int total = row_blocks * q.out_blocks * q.splits;
    int id = q.first + blockIdx.x;
    if (id >= total) return;
    {
        const int xcd = id & 7, each = total >> 3, more = total & 7;
        id = xcd * each + (xcd < more ? xcd : more) + (id >> 3);
    }
    const int blocks = row_blocks * q.out_blocks;
    const int split = id / blocks;
    id -= split * blocks;
    // Neighbours share the weights of up to kRowGroup row blocks of one expert,
    // then its other outputs follow: an L2 reads weights once and the rows of few experts
    // at a time (groups of 16 blocks of whatever expert read 1.6 times the weights' bytes).
    int rb = id / q.out_blocks, g0 = rb / kRowGroup * kRowGroup;
    int high = row_blocks - g0 < kRowGroup ? row_blocks - g0 : kRowGroup;
    if (q.row_list) {
        const int g = q.row_list[1 + rb].group;
        g0 = g >> 5;
        high = g & 31;
    }
    id -= g0 * q.out_blocks;
    rb = g0 + id % high;
    const int tile0 = id / high * OT;

    Span span = {rb * kManyRows, min(rb * kManyRows + kManyRows, a.rows)};
    int f = 0;
    if (q.row_list) {
        const RowBlock b = q.row_list[1 + rb];
        f = b.f;
        span = {b.begin, b.end};
    }
    if (f == a.experts) {  // rows of no expert
        for (int e = threadIdx.x; e < (span.end - span.begin) * OT * 16; e += 256) {
            const int o = tile0 * 16 + e % (OT * 16);
            if (o < a.n) static_cast<T *>(a.y)[(long long)(span.begin + e / (OT * 16)) * a.ldy + o] = (T)0.0f;
        }
        return;
    }
    if (span.end - span.begin > 64) many_rows<DT, 4, NT, WD>(a, q, lds, f, span, tile0, split);
    else if (span.end - span.begin > 32) many_rows<DT, 2, NT, WD>(a, q, lds, f, span, tile0, split);
    else many_rows<DT, 1, NT, WD>(a, q, lds, f, span, tile0, split);
}

// Adds the splits' sums in order.  Bound by its bytes: 4 sums of 256 x 4096, 19 MB, 4.0 to 4.2 us.
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

// Few-row kernels: output tiles, row tiles, waves.
enum FewVariant { k118, k214, k218, k224, k414, k418, k424 };

struct Mx4Plan {
    bool quantise;  // x is quantised by a launch of its own
    int many;       // rows of x a workgroup of the many-row kernel takes; 0: the few-row kernel
    int nt;         // many: blocks of 32 outputs a wave
    FewVariant variant;
    Mx4Many q;
    size_t scales_offset, list_offset, sums_offset, bytes;
};

Mx4Plan plan_mx4(const Mx4Args &a, int dtype, bool given, int cus)
{
    Mx4Plan p{};
    const int mean = (a.rows + a.experts - 1) / a.experts;
    // The few-row kernel reads the codes once for 16 or 32 rows, of one layer or
    // of each expert; the many-row kernel takes 128 rows and its launches cost 5 to
    // 10 us more.  It pays for many codes read that way, and where its workgroups
    // fill half the card without splitting the inputs.  One layer, few against many:
    // 25088 -> 4096, 32 rows 16.6 us and 19.4, 64 rows 22.2 and 20.5; 12000 -> 6000,
    // 40 rows 25.9 and 16.6; 8192 -> 11008, 32 rows 13.7 and 17.3, 48 rows 19.6 and 18.0;
    // 4096 -> 1024, 512 rows 11.0 and 16.0; 512 -> 512, 8192 rows 15.2 and 10.5; 1024 ->
    // 4096, 512 rows 11.2 and 9.5.  Up to 16 rows the codes are read once by either: 16384 ->
    // 16384, 1 row 28.3 and 33.1, 16 rows 29.0 and 33.8; 25088 -> 11008, 1 row 30.6 and 33.4, 16 rows
    // 35.9 and 34.4; 12288 -> 49152, 1 row 56.3 and 60.9, 16 rows 59.5 and 63.6; 32768 -> 32768 within 1%; 17
    // to 32 rows there 31.0 to 31.7 and 33.9 to 35.0; 34.9 to 38.9 and 34.6 to 36.2; 60.1 to 62.4 and 63.8 to 64.7; 16384 ->
    // 8192 25.0 to 25.9 and 22.5 to 23.0.  64 experts of 2048 -> 2816, 16 rows each 34.5 and
    // 39.0, 32 rows each 50.2 and 40.0.
    const long long blocks = (a.rows + 127LL) / 128 * ((a.tiles + 7) / 8);
    const bool many = a.offsets ? mean > 20
                                : (a.rows > 16 && (a.rows + 15LL) / 16 * a.tiles * a.steps * 2048 > 1LL << (a.rows > 32 ? 26 : 27)) ||
                                      (a.rows > 128 && blocks * 2 >= cus);
    p.many = many ? kManyRows : 0;
    // Quantising in the few-row kernel costs every workgroup a little for each step, more
    // in fp32; a launch of its own costs 1.2 to 2 us and the host's call.  There against in
    // a launch, us in a captured graph, weights that are in no cache:
    //   one layer, 4096 and 11008 outputs     bf16                   fp32
    //     1 row, 13 steps                   5.0  6.3   8.0  9.5    5.4 6.0    9.4  9.4
    //     1 row, 16                         5.2  6.2   8.7  9.6    5.9 6.0   10.4  9.4
    //     1 row, 24                         7.5  7.8  11.6 11.6    9.2 8.0   13.6 11.7
    //     1 row, 32                         9.0  8.6  14.4 13.6   11.0 9.0   17.1 13.9
    //     12 rows, 8                        5.0  6.4   7.2  8.2    6.3 6.8    8.5  8.7
    //     8 rows, 13                        5.6  6.6   9.6  9.9    7.9 7.0   11.1 10.3
    //     12 rows, 13                       6.7  6.8  10.6 10.2    9.0 7.1   12.6 10.6
    //     12 rows, 16                       6.8  7.0  11.5 10.5   10.0 7.4   13.9 10.9
    //   of more outputs than the card takes four tiles a compute unit at once
    //     16384: 1 row, 4 and 16 steps      5.0  6.4  10.5 10.8    5.3 6.4   11.7 10.6
    //     17408                             7.3  7.0  15.4 12.8    7.8 7.1   18.4 12.6
    //     65536: 1 row, 1 and 8 steps       9.6  7.3  20.8 16.8   10.1 7.3   23.3 16.8
    //   experts x outputs, rows each, steps
    //     8 x 4096, 1, 8 and 2, 16          9.3 10.2  17.2 17.4   11.4 10.7  19.6 17.9
    //     16 x 1024, 2, 8 and 16            7.8  8.7  12.6 11.5    8.5  9.3  13.7 12.3
    //     8 x 4096, 8 and 12, 8            12.0 13.0  16.8 12.9   14.2 13.4  15.8 13.7
    //     64 x 1024, 8 and 12, 2            9.0 10.9  11.4 11.6   10.5 11.3  14.3 12.0
    //     128 x 1024, 12 and 16, 2         16.8 16.6  19.7 17.8   21.3 17.3  26.4 18.6
    //   the more workgroups, the more of them quantise the same rows: 2 rows each,
    //     16 x 1024, 8 (8192 cells)         7.8  8.7               8.5  9.3
    //     128 x 256, 8 (16384)             10.5 12.2              12.2 12.7
    //     64 x 2816, 2 (22528)             16.4 18.2              21.1 18.3
    //     128 x 1024, 4 (32768)            16.9 18.3              22.2 19.2
    //     128 x 1024, 8 (65536)            28.0 27.0              32.9 27.5
    //     64 x 2816, 8 (90112)             34.2 33.4              44.7 35.6
    // Of 1814 such points the form taken is 0.3% slower than the better one on average,
    // 23% at worst (128 x 256, 12 rows each of 4 steps, fp32: 13.7 and 11.1).
    const bool fp32 = dtype == BCONV_F32;
    const long long cells = (long long)a.experts * a.tiles * a.steps;  // 2 KiB of codes each
    const bool apart = a.offsets ? a.steps > 9 || mean > 12 || mean * a.steps > 64 || cells > (fp32 ? 1 << 13 : 1 << 15)
                                 : a.rows > 16 || a.tiles > 4 * cus || a.steps > (fp32 ? 13 : 20) ||
                                       a.rows * a.steps > (fp32 ? 96 : 160);
    p.quantise = !given && (many || apart);
    auto take = [&](size_t n) {
        const size_t at = p.bytes;
        p.bytes += (n + 255) / 256 * 256;
        return at;
    };
    if (p.quantise) {
        take((size_t)a.x_rows * a.steps * (kStep / 2));
        p.scales_offset = take((size_t)a.x_rows * a.steps * (kStep / 32));
    }
    if (!many) {
        // Output tiles and row tiles a workgroup share their operands, waves the
        // inputs.  One tile and eight waves while that is two workgroups a compute
        // unit at most (16 rows of 25088 -> 4096: 14.1 us, two tiles 16.0; of 2048 ->
        // 16384: two tiles and four waves 7.0, one tile 7.9); more rows share more (32 rows of
        // 8192 -> 11008: four and two tiles 14.3, two tiles 16.7; 128 of 4096 -> 4096: 10.0 and 11.4).
        // Experts: two and two tiles (16 rows each of 8 of 4096 -> 4096: 16.5; four and two 17.1).
        const bool small = a.tiles <= 2 * cus, direct = !given && !p.quantise;
        if (a.offsets) p.variant = direct ? k414 : k224;
        else if (direct) p.variant = small ? k118 : k418;
        else if (a.rows <= 16) p.variant = small ? k118 : k214;
        else if (small && a.rows <= 64) p.variant = a.rows <= 32 ? k218 : k418;
        else p.variant = k424;
        return p;
    }
    p.q.row_blocks = a.offsets ? row_blocks_most(a.rows, a.experts, p.many) : (a.rows + p.many - 1) / p.many;
    // 256 outputs a workgroup where that fills the card (8192 x 8192 -> 8192: 321 us, 128 outputs 382; 16396 rows
    // of 64 experts: 73, 91); otherwise 128 and weights requested three steps ahead (256 x 25088 -> 4096: 28.2, 30.9).
    const long long wide = (long long)p.q.row_blocks * ((a.tiles + 15) / 16);
    p.nt = wide >= cus ? 2 : 1;
    p.q.out_blocks = (a.tiles + p.nt * 8 - 1) / (p.nt * 8);
    p.q.padded_n = p.q.out_blocks * p.nt * 128;
    p.q.splits = 1;
    if (a.offsets) {
        p.list_offset = take((size_t)(p.q.row_blocks + 1) * sizeof(RowBlock));
    } else {
        // a workgroup a compute unit, at least 12 steps each: joining the sums costs 5 us and more (256 x 4096 ->
        // 4096, 16 steps: two splits 15.7, one 13.5; 200 x 8192 -> 2048, 32 steps: two splits 17.2, one 18.9)
        long long splits = cus / ((long long)p.q.row_blocks * p.q.out_blocks);
        if (splits > a.steps / 12) splits = a.steps / 12;
        if (splits > 8) splits = 8;
        if (splits > 1) {
            p.q.splits = (int)splits;
            p.sums_offset = take((size_t)splits * a.rows * p.q.padded_n * 4);
        }
    }
    return p;
}

// Rows that one set of launches takes: one layer's call of more is several, so that
// its quantised rows stay below 2 GiB.
constexpr long long kMaxSteps = 1 << 24;  // rows times steps

int slab_rows(int steps)
{
    const long long rows = kMaxSteps / steps / kManyRows * kManyRows;  // steps <= 2^12
    return (int)(rows < 1 << 18 ? rows : 1 << 18);
}

// The list of row blocks that the plan needs.
RowBlocks row_blocks(const Mx4Args &a, const Mx4Plan &p)
{
    return {a.offsets, const_cast<RowBlock *>(p.q.row_list), a.experts, a.rows, p.many};
}

template <int DT, bool QUANTISED, int RT, int CT, int WAVES> hipError_t run_few(const Mx4Args &a, hipStream_t s)
{
    const dim3 grid((a.tiles + RT - 1) / RT, a.offsets ? a.experts + 1 : (a.rows + 16 * CT - 1) / (16 * CT));
    hipLaunchKernelGGL((mx4_few_kernel<DT, QUANTISED, RT, CT, WAVES>), grid, dim3(WAVES * 64), 0, s, a);
    return hipGetLastError();
}

template <int DT> hipError_t run_mx4(const Mx4Args &a, const Mx4Plan &p, hipStream_t s)
{
    if (p.many) {
        Mx4Many q = p.q;
        const hipError_t e = launch_slices((long long)q.row_blocks * q.out_blocks * q.splits, [&](long long first, unsigned groups) {
            q.first = (int)first;
            if (p.nt == 2) hipLaunchKernelGGL((mx4_many_kernel<DT, 2, 1>), dim3(groups), dim3(256), 0, s, a, q);
            else hipLaunchKernelGGL((mx4_many_kernel<DT, 1, 3>), dim3(groups), dim3(256), 0, s, a, q);
        });
        if (e != hipSuccess || p.q.splits == 1) return e;
        const long long outs = (long long)((a.n + 3) / 4) * a.rows;
        hipLaunchKernelGGL((mx4_join_kernel<DT>), dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, s, a, p.q);
        return hipGetLastError();
    }
    if (a.x) switch (p.variant) {
        case k118: return run_few<DT, false, 1, 1, 8>(a, s);
        case k414: return run_few<DT, false, 4, 1, 4>(a, s);
        default: return run_few<DT, false, 4, 1, 8>(a, s);
        }
    switch (p.variant) {
    case k118: return run_few<DT, true, 1, 1, 8>(a, s);
    case k214: return run_few<DT, true, 2, 1, 4>(a, s);
    case k218: return run_few<DT, true, 2, 1, 8>(a, s);
    case k224: return run_few<DT, true, 2, 2, 4>(a, s);
    case k418: return run_few<DT, true, 4, 1, 8>(a, s);
    default: return run_few<DT, true, 4, 2, 4>(a, s);
    }
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
using bconv::rows_overlap;

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
// Offsets of the many-row kernel into quantised rows are 31 bits; as many rows as
// can be sorted leave room for what int32 counts of rows and their blocks add.
bconv_status_t check_sizes(bconv_mx4_linear_t h, const bconv_mx4_rows_t *args)
{
    if (!h || !args) return fail(BCONV_ERR_INVALID_ARGUMENT, "handle or args is NULL");
    if (args->rows < 0 || args->x_rows < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows and x_rows must be >= 0");
    if (!dtype_bytes(args->dtype)) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", args->dtype);
    if (args->choices < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "choices must be >= 0");
    if (args->choices == 0 ? args->x_rows != args->rows : (long long)args->x_rows * args->choices != args->rows)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "%d rows do not follow from %d input rows and %d choices", args->rows,
                    args->x_rows, args->choices);
    if (!args->offsets && h->desc.experts == 1) return BCONV_OK;  // slabs of rows
    if (args->rows > bconv::kMaxPairs) return fail(BCONV_ERR_INVALID_ARGUMENT, "%d rows of experts are more than 2^27", args->rows);
    if ((long long)args->x_rows * h->steps > bconv::kMaxSteps)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "%d input rows of %d values are more than 2^32 values (padded)", args->x_rows,
                    h->desc.in_features);
    return BCONV_OK;
}

// Workspace of a call: that of its slabs of rows.
size_t workspace_of(bconv_mx4_linear_t h, const bconv::Mx4Args &a, int dtype, bool given)
{
    bconv::Mx4Args part = a;
    const int slab = a.offsets ? a.rows : bconv::slab_rows(a.steps);
    size_t bytes = 0;
    for (const int rows : {a.rows < slab ? a.rows : slab, a.rows % slab}) {
        part.rows = rows;
        part.x_rows = a.offsets ? a.x_rows : rows;
        if (rows == 0) continue;
        const size_t need = bconv::plan_mx4(part, dtype, given, h->cus).bytes;
        bytes = need > bytes ? need : bytes;
    }
    return bytes;
}

bconv::Mx4Args kernel_args(bconv_mx4_linear_t h, const bconv_mx4_rows_t *args)
{
    bconv::Mx4Args a{};
    a.codes = reinterpret_cast<const bconv::u32x4 *>(h->d_codes);
    a.scales = h->d_scales;
    a.bias = h->d_bias;
    a.x = args->x;
    a.xc = args->codes;
    a.xs = args->scales;
    a.xs_row = h->steps * 8LL;
    a.xs_step = 8;
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
    *bytes = args->rows ? workspace_of(h, kernel_args(h, args), args->dtype, !args->x) : 0;
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
    if (args->ldy < n || args->ldy > bconv::kMaxStride) return fail(BCONV_ERR_INVALID_ARGUMENT, "ldy must be in [out_features, 2^30]");
    if (args->x && (args->ldx < k || args->ldx > bconv::kMaxStride))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "ldx must be in [in_features, 2^30]");
    if (((uintptr_t)args->x | (uintptr_t)args->y) % es) return fail(BCONV_ERR_INVALID_ARGUMENT, "x/y not aligned to an element");
    if ((uintptr_t)args->codes % 16 || (uintptr_t)args->scales % 8)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "codes must be 16-byte aligned, scales 8-byte");
    if (!args->offsets && h->desc.experts > 1) return fail(BCONV_ERR_INVALID_ARGUMENT, "offsets is NULL, the layer has experts");
    if ((args->choices > 0) != (args->order != nullptr))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "order must be given with choices, and only then");
    if (args->order && !args->offsets) return fail(BCONV_ERR_INVALID_ARGUMENT, "order is given without offsets");
    if (((uintptr_t)args->offsets | (uintptr_t)args->order) % 4)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "offsets/order not aligned to an element");
    bconv::Mx4Args a = kernel_args(h, args);
    const size_t need = workspace_of(h, a, args->dtype, !args->x);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(BCONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : (size_t)0);
    if (need > 0 && (uintptr_t)workspace % 16) return fail(BCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    const size_t xc = (size_t)args->x_rows * h->steps * (bconv::kStep / 2), xs = xc / 16;
    struct Extent { const void *p; size_t n; };
    const Extent in[] = {
        {args->codes, args->codes ? xc : 0}, {args->scales, args->scales ? xs : 0},
        {args->offsets, args->offsets ? ((size_t)h->desc.experts + 1) * 4 : 0}, {args->order, args->order ? (size_t)args->rows * 4 : 0}};
    const Extent x = {args->x, args->x ? ((size_t)(args->x_rows - 1) * args->ldx + k) * es : 0};
    const Extent out[] = {{args->y, ((size_t)(args->rows - 1) * args->ldy + n) * es}, {workspace, need}};
    bool overlap = x.n && rows_overlap(args->x, args->ldx, k, args->x_rows, args->y, args->ldy, n, args->rows, es);
    overlap = overlap || (x.n && need && ranges_overlap(x.p, x.n, workspace, need));
    for (const auto &o : out)
        for (const auto &i : in) overlap = overlap || (o.n && i.n && ranges_overlap(o.p, o.n, i.p, i.n));
    if (overlap) return fail(BCONV_ERR_INVALID_ARGUMENT, "y or the workspace overlaps x, codes, scales, offsets or order");
    if (need && ranges_overlap(out[0].p, out[0].n, workspace, need))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "y and the workspace overlap");

    DeviceGuard guard(h->device);
    if (guard.err != hipSuccess) return hip_fail(guard.err, "hipSetDevice");
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    const int slab = a.offsets ? a.rows : bconv::slab_rows(a.steps);
    for (int64_t first = 0; first < args->rows; first += slab) {
        if (!a.offsets) {
            a.rows = a.x_rows = (int)(args->rows - first < slab ? args->rows - first : slab);
            a.x = args->x ? static_cast<const char *>(args->x) + first * args->ldx * es : nullptr;
            a.xc = args->codes ? args->codes + first * h->steps * (bconv::kStep / 2) : nullptr;
            a.xs = args->scales ? args->scales + first * h->steps * (bconv::kStep / 32) : nullptr;
            a.y = static_cast<char *>(args->y) + first * args->ldy * es;
        }
        bconv::Mx4Plan p = bconv::plan_mx4(a, args->dtype, !args->x, h->cus);
        p.q.sums = reinterpret_cast<float *>(ws + p.sums_offset);
        if (p.many && a.offsets) p.q.row_list = reinterpret_cast<const bconv::RowBlock *>(ws + p.list_offset);
        hipError_t e = hipSuccess;
        if (p.quantise) {
            uint8_t *codes = reinterpret_cast<uint8_t *>(ws);
            a.xs_row = 8;
            a.xs_step = a.x_rows * 8LL;
            e = bconv::mx4_quantize_rows(s, a.x_rows, k, args->dtype, a.x, a.ldx, codes, codes + p.scales_offset, a.xs_row,
                                         a.xs_step, nullptr, bconv::row_blocks(a, p));
            if (e != hipSuccess) return hip_fail(e, "mx4 quantisation kernel");
            a.x = nullptr;
            a.xc = codes;
            a.xs = codes + p.scales_offset;
        } else if (p.q.row_list) {
            hipLaunchKernelGGL(bconv::mx4_blocks_kernel, dim3(1), dim3(bconv::kListThreads), 0, s, bconv::row_blocks(a, p));
            e = hipGetLastError();
            if (e != hipSuccess) return hip_fail(e, "mx4 row block kernel");
        }
        switch (args->dtype) {
        case BCONV_F32: e = bconv::run_mx4<BCONV_F32>(a, p, s); break;
        case BCONV_F16: e = bconv::run_mx4<BCONV_F16>(a, p, s); break;
        default: e = bconv::run_mx4<BCONV_BF16>(a, p, s); break;
        }
        if (e != hipSuccess) return hip_fail(e, "mx4 linear kernel");
    }
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
