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

#include <new>

#include "host.h"
#include "q4_device.h"

namespace bconv {

constexpr int kChunk = 128;         // inputs of one 16-byte load a lane

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

// Scales and zero points of one output tile and chunk, as a lane uses them:
// the scales of its 4 result rows, and for the codes' zero points either those
// of its result rows (bf16, taken out as a multiple of sum x) or of its operand
// row (fp16 and fp32, subtracted from the codes).
template <int DT, bool ZP, int STEPS> struct Scales {
    static constexpr int N = 4 / STEPS;  // groups a chunk
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    f16x4 s[N];
    uint32_t z[ZP ? N : 1];
    __device__ __forceinline__ void load(const uint16_t *sc, const uint8_t *zp, int lane)
    {
#pragma unroll
        for (int g = 0; g < N; ++g) {
            s[g] = *reinterpret_cast<const f16x4 *>(sc + g * 16 + (lane >> 4) * 4);
            if constexpr (ZP) {
                if constexpr (DT == BCONV_BF16) z[g] = *reinterpret_cast<const uint32_t *>(zp + g * 16 + (lane >> 4) * 4);
                else z[g] = zp[g * 16 + (lane & 15)];
            }
        }
    }
    __device__ __forceinline__ float scale(int g, int i) const { return (float)s[g][i]; }
    __device__ __forceinline__ Zero<DT> zero(int g) const
    {
        if constexpr (ZP && DT != BCONV_BF16) return Zero<DT>((int)z[g]);
        else return Zero<DT>(8);
    }
    // What a group's product starts from: `off` is -24 sum x, or -sum x with
    // zero points.
    __device__ __forceinline__ f32x4 start(int g, float off) const
    {
        if constexpr (DT != BCONV_BF16) return f32x4{0, 0, 0, 0};
        if constexpr (!ZP) return f32x4{off, off, off, off};
        f32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = (float)(16 + ((z[ZP ? g : 0] >> (8 * i)) & 255u)) * off;
        return r;
    }
};

// One chunk (16 RT outputs x 128 inputs) times 16 rows of x, added to acc.
// STEPS: 32-input steps a group.  Per group and output tile the products of one
// group are summed first, then scaled once in fp32; `from` takes the power of
// two of an fp32 row's operands out of the chunk's sum.
template <int DT, bool ZP, int STEPS, int RT>
__device__ __forceinline__ void chunk_product(const u32x4 (&w)[RT], const Operand<DT> (&x)[4],
                                              const Scales<DT, ZP, STEPS> (&sc)[RT], const CodeBits &bits,
                                              float from, f32x4 (&acc)[RT])
{
    constexpr int P = kSplit<DT>;
    f32x4 sum[RT];
    if constexpr (P > 1) {
#pragma unroll
        for (int r = 0; r < RT; ++r) sum[r] = f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int g = 0; g < 4 / STEPS; ++g) {
        // bf16: the offset 16 + z of the codes leaves -(16 + z) sum x, on the
        // matrix cores as well (a constant operand times x), all in units of kUnit
        f32x4 off = {0, 0, 0, 0};
        if constexpr (DT == BCONV_BF16) {
            const u32x4 c = constant<DT>(ZP ? -kUnit<DT> : -24.0f * kUnit<DT>);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) off = mfma_parts<DT>(c, x[g * STEPS + s], off);
        }
        // step by step over all tiles, an fp32 row's parts in sums of their
        // own: a product waits for the one before that adds to the same sum
        f32x4 d[RT][P];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            d[r][0] = ZP ? sc[r].start(g, off[0]) : off;
#pragma unroll
            for (int p = 1; p < P; ++p) d[r][p] = f32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const u32x4 k = decode<DT>(w[r][g * STEPS + s], sc[r].zero(g), bits);
#pragma unroll
                for (int p = 0; p < P; ++p) d[r][p] = mfma16<DT>(k, x[g * STEPS + s].part[p], d[r][p]);
            }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if constexpr (P > 1) d[r][0] += d[r][1];
            f32x4 &to = P > 1 ? sum[r] : acc[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = __builtin_fmaf(sc[r].scale(g, i), d[r][0][i], to[i]);
        }
    }
    if constexpr (P > 1) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][i] = __builtin_fmaf(sum[r][i], from, acc[r][i]);
    }
}

// 4 consecutive outputs of a row (in units of kUnit), with the bias, as far as
// there are outputs.
template <int DT> __device__ __forceinline__ void store_outputs(const Q4Args &a, int m, int o0, f32x4 v)
{
    typedef typename Elem<DT>::type T;
    T *y = static_cast<T *>(a.y) + (long long)m * a.ldy + o0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (o0 + i < a.n) y[i] = round_to<DT>(__builtin_fmaf(v[i], 1.0f / kUnit<DT>, a.bias ? a.bias[o0 + i] : 0.0f));
}

// Few rows of x.  A workgroup takes 16 RT outputs and 16 rows of x; its waves
// split the inputs chunk by chunk and add their sums in LDS, in a fixed order:
// one launch, and with one output tile a workgroup every compute unit has codes
// to stream from about 4096 outputs on.
//
// Bound by the codes' bytes for one row of x (1 x 25088 -> 4096 bf16: 12.4 us for
// 53 MB, 4.3 TB/s with 2.8 us of launch among them; a large read reaches 6.05),
// by x's operands, which every output tile reads again, for 16 rows (29.6 us).
// 13 x 5000 -> 11003 bf16 10.5 us, fp16 10.0; fp32 14.7 us, by the instructions that split x
// (19.8 with exact bf16 codes and three bf16 parts of x; 1 x 25088 -> 4096 26
// against 39).  Requesting a wave's next chunk before working on this one was
// slower (13 rows bf16 13.8 us against 12.3): other waves hide the latency, and
// the registers cost waves.
template <int DT, bool ZP, int STEPS, int RT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void q4_few_kernel(Q4Args a)
{
    typedef typename Elem<DT>::type T;
    constexpr int per_chunk = 4 / STEPS;
    __shared__ f32x4 part[WAVES][RT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile0 = blockIdx.x * RT, m0 = blockIdx.y * 16;
    const int row = lane & 15, lg = lane >> 4;
    const CodeBits bits = code_bits<DT>();

    f32x4 acc[RT];
    long long first[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        acc[r] = f32x4{0, 0, 0, 0};
        first[r] = (long long)(tile0 + r < a.tiles ? tile0 + r : a.tiles - 1) * a.chunks;
    }
    // Lanes of columns past the last row load nothing: their operands stay 0,
    // and their results are not stored.
    const bool real = m0 + row < a.m;
    const T *xr = static_cast<const T *>(a.x) + (real ? (long long)(m0 + row) * a.ldx : 0) + lg * 8;
    Raw<DT> xf[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) xf[s] = zero_raw<DT>();
    const int whole = a.vec ? a.k / kChunk : 0;  // chunks whose columns are 16-byte loads throughout

    for (int c = wave; c < a.chunks; c += WAVES) {
        u32x4 w[RT];
        Scales<DT, ZP, STEPS> sc[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const long long tc = first[r] + c;
            w[r] = *reinterpret_cast<const u32x4 *>(a.codes + tc * 256 + lane * 4);
            sc[r].load(a.scales + tc * per_chunk * 16, ZP ? a.zeros + tc * per_chunk * 16 : nullptr, lane);
        }
        if (real) {
            const T *p = xr + c * kChunk;
            if (c < whole) {
#pragma unroll
                for (int s = 0; s < 4; ++s) xf[s] = load_raw<DT>(p + s * 32);
            } else {
#pragma unroll
                for (int s = 0; s < 4; ++s) xf[s] = load_eight<DT>(p + s * 32, c * kChunk + s * 32 + lg * 8, a.k, a.vec != 0);
            }
        }
        Operand<DT> x[4];
        const float from = to_operands<DT>(xf, x);
        chunk_product<DT, ZP, STEPS, RT>(w, x, sc, bits, from, acc);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) part[wave][r][lane] = acc[r];
    __syncthreads();
    for (int e = threadIdx.x; e < RT * 64; e += WAVES * 64) {
        const int l = e & 63, r = e >> 6;
        const int m = m0 + (l & 15), o0 = (tile0 + r) * 16 + (l >> 4) * 4;
        if (m >= a.m || o0 >= a.n) continue;
        f32x4 v = part[0][r][l];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += part[w][r][l];
        store_outputs<DT>(a, m, o0, v);
    }
}

// ------------------------------------------------------------------ many rows

// What the product of many rows takes besides Q4Args: x laid out as operands
// and the partial sums of the splits.
struct Q4Many {
    u32x4 *xp;       // [column tiles][chunks * 4][parts][64]
    float *xs;       // [column tiles][chunks][groups a chunk][16]; bf16: -sum x (times 24 without zero points), in units,
                     // fp32: the power of two to take out of a group's products
    float *sums;     // [splits][column tiles * 16][padded outputs], or nullptr for one split
    int col_tiles;   // padded to the workgroup's
    int padded_n;
    int row_blocks, col_blocks, splits;
};

// x as operands, a wave a (16 rows, group) pair: converted, split and padded
// with zeros once instead of once per output tile, with the group's sum that
// the codes' offset and zero points multiply.  Bound by its bytes: 256 x 25088
// bf16, 12.8 MB in and out, 6.4 us (4.0 TB/s).
template <int DT, bool ZP, int STEPS>
__global__ __launch_bounds__(256) void q4_pack_kernel(Q4Args a, Q4Many q)
{
    typedef typename Elem<DT>::type T;
    const int lane = threadIdx.x & 63;
    const long long id = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int groups = a.chunks * (4 / STEPS);
    if (id >= (long long)q.col_tiles * groups) return;
    const int g = (int)(id % groups), tile = (int)(id / groups);
    const int m = tile * 16 + (lane & 15);
    Raw<DT> raw[STEPS];
    Operand<DT> o[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int k = (g * STEPS + s) * 32 + (lane >> 4) * 8;
        if (m < a.m && k < a.k)
            raw[s] = load_eight<DT>(static_cast<const T *>(a.x) + (long long)m * a.ldx + k, k, a.k, a.vec != 0);
        else raw[s] = zero_raw<DT>();
    }
    float xs = to_operands<DT>(raw, o);
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        u32x4 *dst = q.xp + ((long long)tile * a.chunks * 4 + g * STEPS + s) * kSplit<DT> * 64 + lane;
#pragma unroll
        for (int p = 0; p < kSplit<DT>; ++p) dst[p * 64] = o[s].part[p];
        if constexpr (DT == BCONV_BF16) sum = mfma_parts<DT>(constant<DT>(ZP ? -kUnit<DT> : -24.0f * kUnit<DT>), o[s], sum);
    }
    if constexpr (DT == BCONV_BF16) xs = sum[0];
    if constexpr (DT != BCONV_F16)
        if (lane < 16) q.xs[((long long)tile * groups + g) * 16 + lane] = xs;
}

// Rows of x a workgroup takes: 128 (64 in fp32, whose operands are two parts),
// or the 64 or 32 that hold them all.
constexpr int most_cols(int dtype) { return dtype == BCONV_F32 ? 64 : 128; }

// Shape of a workgroup of the many-row kernel: its four waves take 64 outputs
// each and, for 32 rows of x, lie along the outputs; otherwise two by two.
template <int COLS> struct ManyShape {
    static constexpr int WC = COLS == 32 ? 1 : 2;     // waves along the rows of x
    static constexpr int CB = COLS / (32 * WC);       // blocks of 32 rows of x a wave
    static constexpr int TILES = 4 / WC * 4;          // output tiles a workgroup
};

// Everything the waves share (the operands and sums of x, scales and zero
// points) goes to LDS a chunk ahead, by loads that pass no registers; the codes
// go to registers, a chunk ahead too.  v_mfma_f32_32x32x16 rather than
// 16x16x32: vector instructions issue beside a matrix instruction for all but
// some 10 of its cycles, whatever its size, and the larger one does twice the
// work in them (measured: 12 vector instructions with one 32x32x16, 58 cycles;
// 6 with one 16x16x32, twice, 68).
//
// Bound by instruction issue: 256 x 25088 -> 4096 bf16, 71 to 74 us (710 to 742 TFLOP/s; a
// large library product reaches 1206), matrix cores busy 39% of the cycles and
// the vector instructions that decode and scale 55%.  Groups of 32 scale four
// times as often as groups of 128: 124 us.  fp32, two products for each,
// with the other two launches: 135 to 142 us (200 with three bf16 parts; bf16 79 to 83,
// fp16 76 to 81).
template <int DT, bool ZP, int STEPS, int COLS>
__global__ __launch_bounds__(256, 2) void q4_many_kernel(Q4Args a, Q4Many q)
{
    typedef ManyShape<COLS> S;
    constexpr int P = kSplit<DT>, G = 4 / STEPS, CB = S::CB, CT = COLS / 16, RT = S::TILES;
    constexpr int UNITS = CT * 4 * P;  // KiB of operands a chunk
    struct Stage {
        u32x4 x[UNITS * 64];
        uint32_t scales[RT * G * 8];                      // [tile][group][16] fp16
        float xs[DT == BCONV_F16 ? 4 : CT * G * 16];      // [column tile][group][16]
        uint32_t zeros[ZP ? RT * G * 4 : 4];              // [tile][group][16] bytes
    };
    __shared__ Stage stage[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 31, half = lane >> 5;
    // Blocks go to the XCDs in turn: the splits of the inputs come first, so
    // that an XCD's L2 sees one slice of x and each code once per column block.
    int id = blockIdx.x;
    const int split = id % q.splits;
    id /= q.splits;
    const int cb0 = id % q.col_blocks, rb0 = id / q.col_blocks;
    const int c_begin = (int)((long long)a.chunks * split / q.splits), c_end = (int)((long long)a.chunks * (split + 1) / q.splits);
    const int tile0 = rb0 * RT, col0 = cb0 * CT;
    const int my_row = wave / S::WC * 4, my_col = wave % S::WC * CB * 2;  // first output and column tile of the wave
    const CodeBits bits = code_bits<DT>();

    auto tile_chunk = [&](int tile, int c) { return (long long)(tile < a.tiles ? tile : a.tiles - 1) * a.chunks + c; };
    typedef __attribute__((address_space(3))) void *Lds;
    auto request = [&](int c) {
        Stage &st = stage[c & 1];
#pragma unroll
        for (int i = 0; i < UNITS / 4; ++i) {
            const int u = i * 4 + wave, t = u / (4 * P), rest = u % (4 * P);
            const u32x4 *src = q.xp + (((long long)(col0 + t) * a.chunks + c) * 4 * P + rest) * 64 + lane;
            __builtin_amdgcn_global_load_lds((const void *)src, (Lds)(&st.x[u * 64]), 16, 0, 0);
        }
        // 4 bytes a lane, the waves in turn; a tile's part of a chunk is consecutive
#pragma unroll
        for (int i = 0; i < (RT * G * 8 + 63) / 64; ++i) {
            const int e = i * 64 + lane;
            if ((i & 3) == wave && e < RT * G * 8) {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(a.scales) +
                                      tile_chunk(tile0 + e / (G * 8), c) * G * 8 + e % (G * 8);
                __builtin_amdgcn_global_load_lds((const void *)src, (Lds)(&st.scales[i * 64]), 4, 0, 0);
            }
        }
        if constexpr (ZP) {
#pragma unroll
            for (int i = 0; i < (RT * G * 4 + 63) / 64; ++i) {
                const int e = i * 64 + lane;
                if (((i + 1) & 3) == wave && e < RT * G * 4) {
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(a.zeros) +
                                          tile_chunk(tile0 + e / (G * 4), c) * G * 4 + e % (G * 4);
                    __builtin_amdgcn_global_load_lds((const void *)src, (Lds)(&st.zeros[i * 64]), 4, 0, 0);
                }
            }
        }
        if constexpr (DT != BCONV_F16) {
#pragma unroll
            for (int i = 0; i < (CT * G * 16 + 63) / 64; ++i) {
                const int e = i * 64 + lane;
                if (((i + 2) & 3) == wave && e < CT * G * 16) {
                    const float *src = q.xs + ((long long)(col0 + e / (G * 16)) * a.chunks + c) * G * 16 + e % (G * 16);
                    __builtin_amdgcn_global_load_lds((const void *)src, (Lds)(&st.xs[i * 64]), 4, 0, 0);
                }
            }
        }
    };
    // Row `row` of a 32 x 16 operand of step (s, j), k = 32 s + 16 j + 8 half on,
    // is word s of lane 16 (2 j + half) + row % 16 of output tile row / 16.
    u32x4 w[2][2], wn[2][2];
    auto fetch = [&](int c) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                wn[r][j] = *reinterpret_cast<const u32x4 *>(
                    a.codes + tile_chunk(tile0 + my_row + r * 2 + (row >> 4), c) * 256 + ((2 * j + half) * 16 + (row & 15)) * 4);
    };
    f32x16 acc[2][CB];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < CB; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[r][t][i] = 0.0f;

    if (c_begin < c_end) {
        request(c_begin);
        fetch(c_begin);
    }
    for (int c = c_begin; c < c_end; ++c) {
        __builtin_amdgcn_s_waitcnt(0 | (0x7 << 4) | (0xf << 8));  // vmcnt(0): this chunk's operands and codes are here
        __syncthreads();                                          // in every wave, and the other stage is read
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) w[r][j] = wn[r][j];
        if (c + 1 < c_end) {
            request(c + 1);
            fetch(c + 1);
        }
        const Stage &st = stage[c & 1];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            // the group's columns stay in registers for the 64 outputs
            u32x4 b[STEPS][2][CB][P];
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int t = 0; t < CB; ++t)
#pragma unroll
                        for (int p = 0; p < P; ++p)
                            b[s][j][t][p] = st.x[(((my_col + t * 2 + (row >> 4)) * 4 + g * STEPS + s) * P + p) * 64 +
                                                 (2 * j + half) * 16 + (row & 15)];
            f32x16 off[CB];  // bf16 without zero points: every sum starts from -24 sum x
            float xs[CB];
#pragma unroll
            for (int t = 0; t < CB; ++t) {
                xs[t] = DT != BCONV_F16 ? st.xs[((my_col + t * 2 + (row >> 4)) * G + g) * 16 + (row & 15)] : 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) off[t][i] = DT == BCONV_BF16 ? xs[t] : 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
                // results 4 v + i are rows 8 v + 4 half + i of the 32
                f16x4 s4[4];
                uint32_t z4[4];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int at = (my_row + r * 2 + (v >> 1)) * G + g, four = (v & 1) * 2 + half;
                    s4[v] = *reinterpret_cast<const f16x4 *>(&st.scales[at * 8 + four * 2]);
                    if constexpr (ZP && DT == BCONV_BF16) z4[v] = st.zeros[at * 4 + four];
                }
                int z = 8;
                if constexpr (ZP && DT != BCONV_BF16)
                    z = reinterpret_cast<const uint8_t *>(st.zeros)[((my_row + r * 2 + (row >> 4)) * G + g) * 16 + (row & 15)];
                const Zero<DT> zero(z);
                f32x16 d[CB];
#pragma unroll
                for (int t = 0; t < CB; ++t) {
                    if constexpr (ZP && DT == BCONV_BF16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) d[t][i] = (float)(16 + ((z4[i >> 2] >> (8 * (i & 3))) & 255u)) * xs[t];
                    } else {
                        d[t] = off[t];
                    }
                }
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const u32x4 k = decode<DT>(w[r][j][g * STEPS + s], zero, bits);
#pragma unroll
                        for (int t = 0; t < CB; ++t)
#pragma unroll
                            for (int p = P - 1; p >= 0; --p) d[t] = mfma32<DT>(k, b[s][j][t][p], d[t]);
                    }
#pragma unroll
                for (int t = 0; t < CB; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float scale = (float)s4[i >> 2][i & 3];
                        // the power of two last: times it alone, the scale could
                        // become subnormal and lose bits
                        if constexpr (DT == BCONV_F32) acc[r][t][i] = __builtin_fmaf(scale * d[t][i], xs[t], acc[r][t][i]);
                        else acc[r][t][i] = __builtin_fmaf(scale, d[t][i], acc[r][t][i]);
                    }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < CB; ++t) {
            const int m = (col0 + my_col + t * 2) * 16 + row;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int o0 = (tile0 + my_row + r * 2) * 16 + v * 8 + half * 4;
                const f32x4 sum = {acc[r][t][4 * v], acc[r][t][4 * v + 1], acc[r][t][4 * v + 2], acc[r][t][4 * v + 3]};
                if (q.splits > 1)
                    *reinterpret_cast<f32x4 *>(q.sums + ((long long)split * q.col_tiles * 16 + m) * q.padded_n + o0) = sum;
                else if (m < a.m && o0 < a.n)
                    store_outputs<DT>(a, m, o0, sum);
            }
        }
}

// Adds the splits' sums in order.  Bound by its bytes: 8 sums of 256 x 4096,
// 35.7 MB, 7.0 us (5.1 TB/s).
template <int DT>
__global__ __launch_bounds__(256) void q4_reduce_kernel(Q4Args a, Q4Many q)
{
    const int per = (a.n + 3) / 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long long)per * a.m) return;
    const int m = (int)(id / per), o0 = (int)(id % per) * 4;
    const float *p = q.sums + (long long)m * q.padded_n + o0;
    const long long step = (long long)q.col_tiles * 16 * q.padded_n;
    f32x4 v = *reinterpret_cast<const f32x4 *>(p);
    for (int s = 1; s < q.splits; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * step);
    store_outputs<DT>(a, m, o0, v);
}

// ------------------------------------------------------------------ dispatch

// Which kernel a number of rows takes, and what it needs of the workspace.
struct Q4Plan {
    bool many;
    int rt, waves;  // few: output tiles and waves a workgroup
    int cols;       // many: rows of x a workgroup
    Q4Many q;
    size_t xs_offset, sums_offset, bytes;
};

// Rows that one set of launches takes: a call of more is several, so that no
// launch passes 32 bits of threads (the packing kernel's waves are (16 rows,
// group) pairs) and the operands' workspace does not grow with the rows for ever.
int slab_rows(int chunks, int per_chunk)
{
    const long long tiles = (1LL << 25) / ((long long)chunks * per_chunk) / 8 * 8;  // chunks * per_chunk <= 2^15
    return tiles < (1 << 14) ? (int)tiles * 16 : 1 << 18;
}

Q4Plan plan_linear(int rows, int dtype, int tiles, int chunks, int per_chunk, int cus)
{
    Q4Plan p{};
    // The few-row kernel reads the codes once for 16 rows of x; the many-row
    // kernel's three launches cost about 8 us more and pay from 32 MiB of codes
    // read that way on (12 in fp32, where the few-row kernel converts x again
    // for every 64 outputs).  bf16, 2048 x 2048: 64 rows 7.0 us against 14.0,
    // 300 rows 25.2 against 23.2; 4096 x 4096: 32 rows 11.2 against 14.5, 128
    // rows 40.3 against 26.8; fp32, 2048 x 2048: 64 rows 11.6 against 16.5, 100
    // rows 19.6 against 17.2; 4096 x 4096: 32 rows 20.0 against 18.1.
    const long long codes = (long long)tiles * chunks;  // KiB
    p.many = rows > 16 && (rows + 15) / 16 * codes > (dtype == BCONV_F32 ? 12288 : 32768);
    if (!p.many) {
        // With several rows, x's operands are shared by as many output tiles as
        // still leave a workgroup for every compute unit (13 x 5000 -> 11003,
        // bf16: four tiles 12.3 us, one 15.0).  One row shares nothing worth it
        // (11.6 against 11.0), except in fp32, which converts it (three tiles 13.6,
        // one 18.8).  Where one tile a workgroup is left and the inputs
        // are long, sixteen waves split them instead of eight (1 x 25088 -> 4096:
        // 12.8 us against 14.6; 1 x 4096 -> 12000: 10.1 against 8.4).
        p.rt = rows > 1 || dtype == BCONV_F32 ? (tiles + cus - 1) / cus : 1;
        if (p.rt > 4) p.rt = 4;
        p.waves = p.rt == 1 && chunks >= 64 && tiles <= 2 * cus ? 16 : 8;
        return p;
    }
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    p.cols = rows <= 32 ? 32 : rows <= 64 ? 64 : most_cols(dtype);
    const int parts = dtype == BCONV_F32 ? 2 : 1;
    const int block_tiles = p.cols == 32 ? ManyShape<32>::TILES : ManyShape<64>::TILES;
    p.q.col_blocks = (rows + p.cols - 1) / p.cols;
    p.q.col_tiles = p.q.col_blocks * (p.cols / 16);
    p.q.row_blocks = (tiles + block_tiles - 1) / block_tiles;
    p.q.padded_n = p.q.row_blocks * block_tiles * 16;
    const long long blocks = (long long)p.q.row_blocks * p.q.col_blocks;
    // two workgroups a compute unit; a slice holds at least 4 chunks
    long long splits = (2LL * cus + blocks - 1) / blocks;
    if (splits > 8) splits = 8;
    if (splits > chunks / 4) splits = chunks / 4;
    p.q.splits = splits < 1 ? 1 : (int)splits;
    p.xs_offset = up((size_t)p.q.col_tiles * chunks * 4 * parts * 1024);
    p.sums_offset = p.xs_offset + (dtype == BCONV_F16 ? 0 : up((size_t)p.q.col_tiles * chunks * per_chunk * 16 * 4));
    p.bytes = p.sums_offset + (p.q.splits > 1 ? (size_t)p.q.splits * p.q.col_tiles * 16 * p.q.padded_n * 4 : 0);
    return p;
}

// The same plan, and workspace, for the last slab's fewer rows.
void fewer_rows(Q4Plan &p, int rows)
{
    if (!p.many) return;
    p.q.col_blocks = (rows + p.cols - 1) / p.cols;
    p.q.col_tiles = p.q.col_blocks * (p.cols / 16);
}

template <int DT, bool ZP, int STEPS, int RT, int WAVES>
hipError_t run_few(const Q4Args &a, hipStream_t s)
{
    const dim3 grid((a.tiles + RT - 1) / RT, (a.m + 15) / 16);
    hipLaunchKernelGGL((q4_few_kernel<DT, ZP, STEPS, RT, WAVES>), grid, dim3(WAVES * 64), 0, s, a);
    return hipGetLastError();
}

template <int DT, bool ZP, int STEPS>
hipError_t run_linear(const Q4Args &a, const Q4Plan &p, hipStream_t s)
{
    if (p.many) {
        const long long packs = (long long)p.q.col_tiles * a.chunks * (4 / STEPS);
        hipLaunchKernelGGL((q4_pack_kernel<DT, ZP, STEPS>), dim3((unsigned)((packs + 3) / 4)), dim3(256), 0, s, a, p.q);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const long long blocks = (long long)p.q.row_blocks * p.q.col_blocks * p.q.splits;
        const dim3 grid((unsigned)blocks);
        if (p.cols == 32)
            hipLaunchKernelGGL((q4_many_kernel<DT, ZP, STEPS, 32>), grid, dim3(256), 0, s, a, p.q);
        else if (p.cols == 64)
            hipLaunchKernelGGL((q4_many_kernel<DT, ZP, STEPS, 64>), grid, dim3(256), 0, s, a, p.q);
        else
            hipLaunchKernelGGL((q4_many_kernel<DT, ZP, STEPS, most_cols(DT)>), grid, dim3(256), 0, s, a, p.q);
        e = hipGetLastError();
        if (e != hipSuccess || p.q.splits == 1) return e;
        const long long outs = (long long)((a.n + 3) / 4) * a.m;
        hipLaunchKernelGGL((q4_reduce_kernel<DT>), dim3((unsigned)((outs + 255) / 256)), dim3(256), 0, s, a, p.q);
        return hipGetLastError();
    }
    switch (p.rt) {
    case 1:
        if (p.waves == 16) return run_few<DT, ZP, STEPS, 1, 16>(a, s);
        return run_few<DT, ZP, STEPS, 1, 8>(a, s);
    case 2: return run_few<DT, ZP, STEPS, 2, 8>(a, s);
    case 3: return run_few<DT, ZP, STEPS, 3, 8>(a, s);
    default: return run_few<DT, ZP, STEPS, 4, 8>(a, s);
    }
}

template <int DT, bool ZP>
hipError_t dispatch_group(const Q4Args &a, const Q4Plan &p, int group, hipStream_t s)
{
    switch (group) {
    case 32: return run_linear<DT, ZP, 1>(a, p, s);
    case 64: return run_linear<DT, ZP, 2>(a, p, s);
    default: return run_linear<DT, ZP, 4>(a, p, s);
    }
}

template <int DT>
hipError_t dispatch_zero(const Q4Args &a, const Q4Plan &p, int group, hipStream_t s)
{
    return a.zeros ? dispatch_group<DT, true>(a, p, group, s) : dispatch_group<DT, false>(a, p, group, s);
}

}  // namespace bconv

struct bconv_q4_linear {
    bconv_q4_linear_desc_t desc;
    int device, cus;
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

// Whether rows of x (k wide, ldx apart) and of y (n wide, ldy apart) share an
// element.  Columns of one buffer (equal strides) lie inside each other's
// extent without sharing any.
bool rows_overlap(const void *x, int64_t ldx, int k, const void *y, int64_t ldy, int n, int rows, int es)
{
    const size_t xb = ((size_t)(rows - 1) * ldx + k) * es, yb = ((size_t)(rows - 1) * ldy + n) * es;
    if (!ranges_overlap(x, xb, y, yb)) return false;
    const intptr_t apart = (intptr_t)((uintptr_t)y - (uintptr_t)x);
    if (ldx != ldy || apart % es) return true;
    int64_t d = apart / es % ldx;  // y's first column among x's
    if (d < 0) d += ldx;
    return d < k || d + n > ldx;
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
    if (e == hipSuccess) e = hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, h->device);
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
    const int slab = bconv::slab_rows(h->chunks, h->per_chunk);
    *bytes = rows ? bconv::plan_linear(rows < slab ? rows : slab, dtype, h->tiles, h->chunks, h->per_chunk, h->cus).bytes : 0;
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
    if (rows_overlap(x, ldx, k, y, ldy, n, rows, es)) return fail(BCONV_ERR_INVALID_ARGUMENT, "x and y overlap");
    const int slab = bconv::slab_rows(h->chunks, h->per_chunk);
    bconv::Q4Plan p = bconv::plan_linear(rows < slab ? rows : slab, dtype, h->tiles, h->chunks, h->per_chunk, h->cus);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes))
        return fail(BCONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    if (p.bytes > 0) {
        if ((uintptr_t)workspace % 16) return fail(BCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
        if (ranges_overlap(workspace, p.bytes, x, xb) || ranges_overlap(workspace, p.bytes, y, yb))
            return fail(BCONV_ERR_INVALID_ARGUMENT, "workspace overlaps x or y");
        char *ws = static_cast<char *>(workspace);
        p.q.xp = reinterpret_cast<bconv::u32x4 *>(ws);
        p.q.xs = reinterpret_cast<float *>(ws + p.xs_offset);
        p.q.sums = reinterpret_cast<float *>(ws + p.sums_offset);
    }

    DeviceGuard guard(h->device);
    if (guard.err != hipSuccess) return hip_fail(guard.err, "hipSetDevice");
    bconv::Q4Args a{};
    a.codes = h->d_codes;
    a.scales = h->d_scales;
    a.zeros = h->d_zeros;
    a.bias = h->d_bias;
    a.ldx = ldx;
    a.ldy = ldy;
    a.n = n;
    a.k = k;
    a.tiles = h->tiles;
    a.chunks = h->chunks;
    a.vec = ((uintptr_t)x % 16 == 0) && (ldx * es % 16 == 0);
    hipStream_t s = static_cast<hipStream_t>(stream);
    for (int64_t first = 0; first < rows; first += slab) {
        a.x = static_cast<const char *>(x) + first * ldx * es;
        a.y = static_cast<char *>(y) + first * ldy * es;
        a.m = (int)(rows - first < slab ? rows - first : slab);
        if (first > 0) bconv::fewer_rows(p, a.m);
        hipError_t e;
        switch (dtype) {
        case BCONV_F32: e = bconv::dispatch_zero<BCONV_F32>(a, p, h->desc.group, s); break;
        case BCONV_F16: e = bconv::dispatch_zero<BCONV_F16>(a, p, h->desc.group, s); break;
        default: e = bconv::dispatch_zero<BCONV_BF16>(a, p, h->desc.group, s); break;
        }
        if (e != hipSuccess) return hip_fail(e, "4-bit linear kernel");
    }
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
