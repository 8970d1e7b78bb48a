// Attention over the paged 4-bit cache: one pass over the keys and values with
// a running softmax, all products on the matrix cores straight from the codes.
//
// For one request and key/value head, the columns of a product are (query,
// head of the group) pairs, 16 a tile, and its rows are tokens (S = K Q^T) or
// channels (O = V^T P).  A wave takes 32 tokens at a time:
//
//   S[t][c] = sum_g s_tg (sum_{d in g} (code - 8) q_d) + b_tg sum_{d in g} q_d
//   O[d][c] += sum_t (code_td - 8) (p_tc s_tg) + sum_t p_tc b_tg
//
// so a key's step scales a finished product and a value's step goes into the
// probability before it is rounded for the matrix cores; the midpoints never
// meet the matrix cores and stay in fp32.  Rows of the first product are
// numbered so that a lane ends up with the probabilities of the 8 tokens whose
// codes it decodes for the second: P never leaves its registers.
//
// Bound by instruction issue, not by the cache's bytes: 128 channels in groups
// of 64 take about 350 vector and 24 matrix instructions a tile (decoding 120,
// steps and midpoints 128, softmax 40) for 4.6 KB, 270 vector ones where few
// columns share their softmax (see Steps).  32 requests of up to 8192 tokens, 32
// heads over 8, bf16: 46.3 us for 183 MB (4.0 TB/s; a large read reaches 6.05), and
// 5.6 us for the join of their parts (all of 8192 tokens: 4.4 TB/s with the join); the
// rest is the requests' uneven lengths and a workgroup's first loads.  Two requests of
// 131071 tokens, 16 heads over one, fp16: 15.4 us and 5.2 us for the join (floor
// 5.5 us).  Four prompts of up to 512 tokens behind up to 2048, 32 heads over 8: 149 us
// in bf16, 176 in fp16 (floor 32.9): each 16 columns decode the same keys and values
// anew.  One token of 777: 7.0 us, a chain of loads (lengths, block ids, keys,
// values).  Registers decide the rest: 128 a wave and four waves a SIMD; spilling
// 15 of them costs 58 -> 84 us, three waves at 168 registers 66.
#include <hip/hip_runtime.h>

#include <cmath>

#include "internal.h"
#include "kv4.h"

namespace bconv {

constexpr int kTokens = 32;       // tokens a wave takes at a time
constexpr int kCols = 16;         // (query, head) columns a workgroup takes
constexpr float kLowest = -3e38f; // running maximum before the first visible token
// How far a logit (base 2) may pass the running maximum before the sums are
// rescaled: 2^8 of headroom costs fp32 sums nothing and saves most rescales.
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnArgs {
    const char *pool;
    const void *q;
    long long q_token, q_head;
    void *out;
    float *lse;
    const int *table, *context, *q_start;
    int requests, q_tokens, max_q, heads, ratio;
    FastDiv by_ratio;
    int width;
    long long stride;
    int max_context, window;
    float scale_log2;  // |scale| log2 e
    uint32_t flip;     // sign bits to flip in q: those of a negative scale
    int vec;
    int col_blocks, parts, part_tokens;  // part_tokens: a multiple of kTokens
    float *part_o;                       // [column rows][parts][dim_padded]
    float2 *part_ml;                     // [column rows][parts]
    Kv4Geom g;
    int first;  // number of the launch's first workgroup
};

constexpr int kMaxParts = 512;

// The columns one workgroup takes and the tokens they see.
struct Span {
    int q0, n, j0, c0, c1;   // first query row, queries, first query's index, columns [c0, c1)
    int last;                // position of the request's query 0 (context - queries)
    int t0, t1;              // tokens [t0, t1), t0 a multiple of kTokens
    int low;                 // the first of them that any column sees
};

__device__ __forceinline__ int first_seen(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

__device__ __forceinline__ Span column_span(const AttnArgs &a, int req, int cb)
{
    Span s;
    int q0, n;
    if (a.q_start) {
        q0 = a.q_start[req];
        n = a.q_start[req + 1] - q0;
    } else {
        n = a.q_tokens / a.requests;
        q0 = req * n;
    }
    const int ctx = a.context[req] > 0 ? a.context[req] : 0;
    if (n < 0) n = 0;
    s.last = ctx - n;
    if (n > a.max_q) n = a.max_q;
    if (q0 < 0 || q0 > a.q_tokens) n = 0;
    else if (n > a.q_tokens - q0) n = a.q_tokens - q0;
    s.q0 = q0;
    s.n = n;
    s.c0 = cb * kCols;
    const int cols = s.n * a.ratio;
    s.c1 = s.c0 + kCols < cols ? s.c0 + kCols : cols;
    s.t0 = s.t1 = s.low = 0;
    s.j0 = 0;
    if (s.c0 < s.c1) {
        s.j0 = (int)fastdiv((uint32_t)s.c0, a.by_ratio);
        const int j1 = (int)fastdiv((uint32_t)(s.c1 - 1), a.by_ratio);
        const int hi = s.last + j1;
        s.t1 = (hi < a.max_context - 1 ? hi : a.max_context - 1) + 1;
        s.low = first_seen(s.last + s.j0, a.window);
        s.t0 = s.low & ~(kTokens - 1);
        // nothing to see: from 0, so that no part's first token passes 32 bits
        if (s.t1 <= s.t0) s.t0 = s.t1 = 0;
    }
    return s;
}

__device__ __forceinline__ float lane_groups_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}

__device__ __forceinline__ float lane_groups_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Type of the operands of V^T P, and parts that a probability, times its value's
// step, is rounded into: one fp16 (11 bits) for bf16 results, two bf16 (16 bits) for
// fp16 results, two fp16 (23 bits) for fp32 results.
//
// fp16's exponents need these products near 1.
//   bf16 results: they are taken times 2^lead, a lead that a wave chooses by the
//     largest step it has met, so that no product passes 2^14; it changes when a
//     larger step comes.  A new maximum's largest product is 2^5 to 2^6, so steps
//     down to 2^-19 of the largest keep all 11 bits, down to 2^-22 the 8 that a
//     bf16 part would.  The lead is added to a logit's distance from the maximum,
//     which is exact where it matters, and not taken off the maximum itself: from
//     2^26 on that would round to more than the lead, and products to infinity.
//     One bf16 part costs the same and adds an error as large as the result's own
//     rounding (2.4e-3 against 1.7e-3 on 32 ragged requests).
//   fp32 results: they are taken times a power of two a column and group of
//     channels, which is chosen anew when the column's maximum moves or a product
//     would pass fp16's largest.  The products stay below 2^(kUnitBits + 1) at a
//     choice and have room to grow until the next.  Against three bf16 parts and
//     exact bf16 codes, for keys as well: 32 requests of up to 8192 tokens, 32
//     heads over 8, 88 -> 72 us; 64 heads 108 -> 87.
// fp16 results gain nothing from either (64 heads: 74 us with bf16 parts, 80 with
// fp16).
template <int DT> constexpr int kValueType = DT == BCONV_F16 ? BCONV_BF16 : BCONV_F16;
template <int DT> constexpr int kProbParts = DT == BCONV_BF16 ? 1 : 2;
constexpr int kUnitBits = 8;
typedef Range<kUnitBits, -40> Unit;  // so that a change of unit keeps fp32 sums in range

// The lead for steps below fp16 `limit` = e << 10, that is below 2^(e - 15): times
// them, probabilities of up to 2^(kSlack + lead) stay up to 2^14.
__device__ __forceinline__ float lead_of(uint32_t limit) { return 29.0f - kSlack - (float)(limit >> 10); }

// A value code decodes to 128 + c in bf16 or 1024 + c in fp16, with no shift for
// the first code.  For fp32 results 1032 is subtracted at once; for fp16 results a
// product with the constant -136 goes with each product, so that the running sums
// hold code - 8 as well and never grow with the offset.  For bf16 results, whose own
// rounding hides what the offset costs an fp32 sum, the sums of the probabilities
// are kept instead (one product a group in place of one a channel tile) and taken
// out at the end: 128 channels in one group, 32 requests of up to 8192 tokens 51.9
// -> 50.3 us.  With two groups the sums' registers would spill (58.3 -> 65.2 us).
constexpr bool sums_probs(int dt, int dp, int groups) { return dt == BCONV_BF16 && !(dp == 128 && groups == 2); }
template <int DT> constexpr float kValueOffset = DT == BCONV_F16 ? 136.0f : 1032.0f;

// The word that lane N of each 16 lanes holds.
template <int N> __device__ __forceinline__ uint32_t from_lane(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + N, 0xf, 0xf, true);
}

// from_lane() of entry e of a table kept 16 entries a register, one a lane: a
// broadcast inside the 16 lanes, so a table costs them one register and one
// load instead of 16.
template <int R> __device__ __forceinline__ uint32_t entry(const uint32_t (&v)[R], int e)
{
    switch (e & 15) {
    case 0: return from_lane<0>(v[e >> 4]);
    case 1: return from_lane<1>(v[e >> 4]);
    case 2: return from_lane<2>(v[e >> 4]);
    case 3: return from_lane<3>(v[e >> 4]);
    case 4: return from_lane<4>(v[e >> 4]);
    case 5: return from_lane<5>(v[e >> 4]);
    case 6: return from_lane<6>(v[e >> 4]);
    case 7: return from_lane<7>(v[e >> 4]);
    case 8: return from_lane<8>(v[e >> 4]);
    case 9: return from_lane<9>(v[e >> 4]);
    case 10: return from_lane<10>(v[e >> 4]);
    case 11: return from_lane<11>(v[e >> 4]);
    case 12: return from_lane<12>(v[e >> 4]);
    case 13: return from_lane<13>(v[e >> 4]);
    case 14: return from_lane<14>(v[e >> 4]);
    default: return from_lane<15>(v[e >> 4]);
    }
}

// Codes j of two tokens' rows (16 bits of each row's part) as a pair.
template <int DT> __device__ __forceinline__ uint32_t value_pair(uint32_t two, int j, const CodeBits &bits)
{
    const uint32_t c = bits(two >> (4 * j));
    if constexpr (DT != BCONV_F32) return c;
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, c) - f16x2{(_Float16)1032.0f, (_Float16)1032.0f});
}

template <int DT> __device__ __forceinline__ CodeBits value_bits()
{
    return opaque_bits(0x000f000fu, kValueType<DT> == BCONV_BF16 ? 0x43004300u : 0x64006400u);  // bf16 128, fp16 1024
}

// Where a lane's part of 32 tokens is.  Runs of 8 tokens never cross a block,
// and the 32 tokens from t, a multiple of 32, lie in at most two: `first` and
// `second` are the records of tokens t and t + 16 for the head.  Row r of S
// tile u is token t + 8 (r / 4) + 4 u + r % 4: a lane's eight results are the run
// of 8 tokens from t + 8 (lane / 16), whose values it decodes.
struct Place {
    const char *first, *second;
    int at;  // token t in its block (0 where a block ends inside the tile)
};

template <int GROUPS> constexpr int kTable = (8 * GROUPS + 15) / 16;

// Where a workgroup has at most four columns, each stands REP = 4 times next to
// itself in the 16, and its copies share its softmax, three quarters of whose
// lanes would be idle: of a run of 8 tokens, numbered 4 u + i, copy r takes those
// with i % REP == r.  It reads their (s, b) itself.
template <int GROUPS, int REP> struct Steps {
    static constexpr int E = 4 / REP;
    uint32_t v[2][E][GROUPS];
    // `t`: the run's (s, b) table
    __device__ __forceinline__ void load(const char *t, int lane)
    {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const char *at = t + (4 * u + e * REP + lane % REP) * GROUPS * 4;
                if constexpr (GROUPS == 1) {
                    v[u][e][0] = *reinterpret_cast<const uint32_t *>(at);
                } else {
#pragma unroll
                    for (int g = 0; g < GROUPS; g += 2) {
                        const u32x2 x = *reinterpret_cast<const u32x2 *>(at + 4 * g);
                        v[u][e][g] = x[0];
                        v[u][e][g + 1] = x[1];
                    }
                }
            }
    }
    __device__ __forceinline__ f16x2 at(int u, int e, int g) const { return __builtin_bit_cast(f16x2, v[u][e][g]); }
    // the largest step's bits among the lane's
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t t = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) t = max(t, v[u][e][g] & 0xffffu);
        return t;
    }
    // drops the tokens that `keep` (of a token's number in the run) denies
    template <typename F> __device__ __forceinline__ void mask(int lane, F keep)
    {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (!keep(4 * u + e * REP + lane % REP)) {
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) v[u][e][g] = 0;
                }
    }
};

// One copy reads every token's: 16 lanes share the run's table, an entry (token
// * GROUPS + group) a lane.
template <int GROUPS> struct Steps<GROUPS, 1> {
    static constexpr int E = 4;
    uint32_t v[kTable<GROUPS>];
    __device__ __forceinline__ static int entry_of(int lane, int x) { return (x * 16 + (lane & 15)) & (8 * GROUPS - 1); }
    __device__ __forceinline__ void load(const char *t, int lane)
    {
#pragma unroll
        for (int x = 0; x < kTable<GROUPS>; ++x) v[x] = *reinterpret_cast<const uint32_t *>(t + entry_of(lane, x) * 4);
    }
    __device__ __forceinline__ f16x2 at(int u, int e, int g) const
    {
        return __builtin_bit_cast(f16x2, entry(v, (4 * u + e) * GROUPS + g));
    }
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t t = v[0] & 0xffffu;
#pragma unroll
        for (int x = 1; x < kTable<GROUPS>; ++x) t = max(t, v[x] & 0xffffu);
        return t;
    }
    template <typename F> __device__ __forceinline__ void mask(int lane, F keep)
    {
#pragma unroll
        for (int x = 0; x < kTable<GROUPS>; ++x)
            if (!keep(entry_of(lane, x) / GROUPS)) v[x] = 0;
    }
};

// Result e of a copy: of the four results of a product, number e REP + r.
template <int REP> __device__ __forceinline__ float own(f32x4 d, int e, int lane)
{
    if constexpr (REP == 1) return d[e];
    const float even = lane & 1 ? d[1] : d[0], odd = lane & 1 ? d[3] : d[2];
    return lane & 2 ? odd : even;
}

// A word of copy r of the lane's column.
template <int REP> __device__ __forceinline__ uint32_t from_copy(uint32_t v, int r)
{
    if constexpr (REP == 1) return v;
    switch (r) {  // the same lane of each four
    case 0: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x00, 0xf, 0xf, true);
    case 1: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x55, 0xf, 0xf, true);
    case 2: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xaa, 0xf, 0xf, true);
    default: return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xff, 0xf, 0xf, true);
    }
}

template <int REP> __device__ __forceinline__ float copies_max(float v)
{
    if constexpr (REP == 1) return v;
    v = fmaxf(v, __shfl_xor(v, 1));
    return fmaxf(v, __shfl_xor(v, 2));
}

template <int REP> __device__ __forceinline__ float copies_sum(float v)
{
    if constexpr (REP == 1) return v;
    v += __shfl_xor(v, 1);
    return v + __shfl_xor(v, 2);
}

// Keys of 32 tokens: words of the lane's two operand rows, and (s, b) of its run.
template <int DP, int GROUPS, int REP> struct Keys {
    uint32_t w[2][DP / 32];
    Steps<GROUPS, REP> steps;
    __device__ __forceinline__ void load(const AttnArgs &a, const Place &p, int lane)
    {
        const int row = lane & 15, lg = lane >> 4, mask = (1 << a.g.block_shift) - 1;
        const char *krec = row & 8 ? p.second : p.first, *trec = lg & 2 ? p.second : p.first;
        const char *k = krec + (p.at + ((row >> 2) * 8 & mask) + (row & 3)) * (DP / 2) + lg * (DP / 8);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if constexpr (DP == 64) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(k + u * 4 * (DP / 2));
                w[u][0] = x[0];
                w[u][1] = x[1];
            } else {
#pragma unroll
                for (int v = 0; v < DP / 128; ++v) {
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(k + u * 4 * (DP / 2) + 16 * v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[u][4 * v + i] = x[i];
                }
            }
        }
        steps.load(trec + a.g.k_scales + (p.at + (lg * 8 & mask)) * GROUPS * 4, lane);
    }
};

// Values of the lane's run: its part of each row (16 bits for DP = 64), and (s, b).
template <int DP, int GROUPS, int REP> struct Values {
    static constexpr int N = DP < 128 ? 1 : DP / 128;
    uint32_t w[8][N];
    Steps<GROUPS, REP> steps;
    __device__ __forceinline__ void load(const AttnArgs &a, const Place &p, int lane)
    {
        const int row = lane & 15, lg = lane >> 4, mask = (1 << a.g.block_shift) - 1;
        const char *rec = lg & 2 ? p.second : p.first;
        const int at = p.at + (lg * 8 & mask);
        steps.load(rec + a.g.v_scales + at * GROUPS * 4, lane);
        const char *v = rec + a.g.v_codes + at * (DP / 2) + row * (DP / 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DP == 64) {
                w[i][0] = *reinterpret_cast<const uint16_t *>(v + i * (DP / 2));
            } else if constexpr (DP == 128) {
                w[i][0] = *reinterpret_cast<const uint32_t *>(v + i * (DP / 2));
            } else {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(v + i * (DP / 2));
                w[i][0] = x[0];
                w[i][1] = x[1];
            }
        }
    }
};

// Waves that share a part of a request's tokens: eight, or four where eight (at
// most 256 registers a wave) would spill.
constexpr int attn_waves(int dt, int dp, int groups) { return dp <= 128 || (groups == 2 && dt != BCONV_F32) ? 8 : 4; }

// Waves a SIMD that the registers are held to.
constexpr int min_waves(int dt, int dp, int groups)
{
    if (dp == 256 || dt == BCONV_F32) return 1;
    return groups >= 4 ? 2 : 4;
}

// FULL: no group of channels is padding alone (such groups are skipped).
// REP: copies of a column (see Steps).
template <int DT, int DP, int GROUPS, bool FULL, int REP>
__global__ __launch_bounds__(attn_waves(DT, DP, GROUPS) * 64, min_waves(DT, DP, GROUPS)) void
kv4_attention_kernel(AttnArgs a)
{
    typedef typename Elem<DT>::type T;
    constexpr int STEPS = DP / 32;             // 32-channel steps of K Q^T
    constexpr int PER = STEPS / GROUPS;        // steps a group
    constexpr int TILES = DP / 16;             // 16-channel tiles of V^T P
    constexpr int VPER = TILES / GROUPS;       // of them a group
    constexpr int NP = kProbParts<DT>, VT = kValueType<DT>;
    constexpr bool UNITS = DT == BCONV_F32, LEAD = DT == BCONV_BF16;
    constexpr int WAVES = attn_waves(DT, DP, GROUPS), COLS = kCols / REP;
    constexpr int E = 4 / REP;                 // tokens of four that a copy takes
    constexpr bool SUMS = sums_probs(DT, DP, GROUPS);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, lg = lane >> 4, col = row / REP;
    int id = a.first + (int)blockIdx.x;
    const int part = id % a.parts;
    id /= a.parts;
    const int cb = id % a.col_blocks;
    id /= a.col_blocks;
    const int head = id % a.g.kv_heads, req = id / a.g.kv_heads;
    // Block ids are the same for a wave's 32 tokens (two of them where blocks are
    // 16 tokens), so they and the records' addresses stay in scalar registers.
    const int *table = a.table + req * a.stride;
    auto block_of = [&](int pos) {
        const int b = pos >> a.g.block_shift;
        return __builtin_amdgcn_readfirstlane(b < a.width ? table[b] : -1);
    };
    // Without a window the part's tokens follow from its number: the first ids
    // are read together with the lengths instead of after them.
    int next0 = -1, next1 = -1;  // block ids of the next tile
    if (a.window == 0) {
        next0 = block_of(part * a.part_tokens + wave * kTokens);
        next1 = block_of(part * a.part_tokens + wave * kTokens + 16);
    }
    const Span sp = column_span(a, req, cb);
    if (sp.c0 >= sp.c1) return;
    const int span = sp.t1 - sp.t0;
    const int begin = sp.t0 + part * a.part_tokens;
    if (part > 0 && begin >= sp.t1) return;
    const int end = begin + a.part_tokens < sp.t1 ? begin + a.part_tokens : sp.t1;
    const bool whole = span <= a.part_tokens;

    // A block that does not exist is read as the pool's first and masked.
    const char *pool = a.pool + (long long)head * a.g.record_bytes;
    const unsigned block_bytes = (unsigned)a.g.kv_heads * (unsigned)a.g.record_bytes;  // below 2^29
    auto exists = [&](int block) { return (unsigned)block < (unsigned)a.g.num_blocks; };
    auto record = [&](int block) { return pool + (unsigned long long)(exists(block) ? (unsigned)block : 0u) * block_bytes; };
    auto place_of = [&](int pos, int b0, int b1) {
        return Place{record(b0), record(b1), pos & ((1 << a.g.block_shift) - 1)};
    };
    constexpr int STRIDE = WAVES * kTokens;
    int t = begin + wave * kTokens;
    Keys<DP, GROUPS, REP> next;
    if (t < end) {
        if (a.window) {
            next0 = block_of(t);
            next1 = block_of(t + 16);
        }
        next.load(a, place_of(t, next0, next1), lane);
    }

    // this lane's columns: row of q, positions seen
    Operand<DT> qf[STEPS];
    float scale = a.scale_log2 * (1.0f / kUnit<DT>);
    int lo, hi;
    int all_lo = 0, all_hi = 0x7fffffff;  // seen by every column
    {
        const int c = sp.c0 + col;
        lo = 0;
        hi = -1;
        const bool real = c < sp.c1;
        const int j = real ? (int)fastdiv((uint32_t)c, a.by_ratio) : 0, h = head * a.ratio + (real ? c - j * a.ratio : 0);
        if (real) {
            const int pos = sp.last + j;
            lo = first_seen(pos, a.window);
            hi = pos < a.max_context ? pos : a.max_context - 1;
            all_lo = lo > all_lo ? lo : all_lo;
            all_hi = hi < all_hi ? hi : all_hi;
        }
        const T *q = static_cast<const T *>(a.q) + (long long)(sp.q0 + j) * a.q_token + (long long)h * a.q_head;
        Raw<DT> raw[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int d = s * 32 + lg * 8;
            if (real && d < a.g.dim) raw[s] = load_eight<DT>(q + d, d, a.g.dim, a.vec != 0);
            else raw[s] = zero_raw<DT>();
        }
        scale *= to_operands<DT>(raw, qf);
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int p = 0; p < kSplit<DT>; ++p) qf[s].part[p] ^= a.flip;
    }
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
        all_lo = max(all_lo, __shfl_xor(all_lo, d));
        all_hi = min(all_hi, __shfl_xor(all_hi, d));
    }
    all_lo = __builtin_amdgcn_readfirstlane(all_lo);
    all_hi = __builtin_amdgcn_readfirstlane(all_hi);

    // sums of q over each group, for the midpoints and the codes' offset (16 in
    // bf16: a product gets -24 of them once it is a lane's own, which takes fewer
    // registers than starting from them), in units of kUnit as the products are
    float qsum[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        f32x4 x = {0, 0, 0, 0};
        const u32x4 one = constant<DT>(kUnit<DT>);
#pragma unroll
        for (int s = 0; s < PER; ++s) x = mfma_parts<DT>(one, qf[g * PER + s], x);
        qsum[g] = x[0];
    }

    f32x4 acc[TILES], psum[SUMS ? GROUPS : 1];
    float mid[GROUPS], m = kLowest, l = 0.0f;
    float unit[UNITS ? GROUPS : 1];  // what the group's products are multiplied by
    // LEAD: steps' bits stay below `limit`, probabilities are times 2^lead
    uint32_t limit = LEAD ? 0u : 1u;
    float lead = 0.0f;
#pragma unroll
    for (int k = 0; k < TILES; ++k) acc[k] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        mid[g] = 0.0f;
        if constexpr (UNITS) unit[g] = 1.0f;
        if constexpr (SUMS) psum[g] = f32x4{0, 0, 0, 0};
    }
    const Zero<DT> eight(8);
    const u32x4 offset = constant<VT>(SUMS ? 1.0f : -kValueOffset<DT>);
    const CodeBits kbits = code_bits<DT>(), vbits = value_bits<DT>();

    const int vrun = lg * 8;
    for (; t < end; t += STRIDE) {
        // the tile's values are requested now and used after the softmax, the
        // next tile's keys a tile ahead
        const int id0 = next0, id1 = next1;
        const Keys<DP, GROUPS, REP> keys = next;
        Values<DP, GROUPS, REP> values;
        values.load(a, place_of(t, id0, id1), lane);
        if (t + STRIDE < end) {
            next0 = block_of(t + STRIDE);
            next1 = block_of(t + STRIDE + 16);
            next.load(a, place_of(t + STRIDE, next0, next1), lane);
        }

        // S; times scale_log2 (a negative scale is in q) these are base-2 logits
        float z[2][E];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) z[u][e] = 0.0f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            if (!FULL && g * PER * 32 >= a.g.dim) continue;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                f32x4 d = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < PER; ++s) {
                    const u32x4 k = decode<DT>(keys.w[u][g * PER + s], eight, kbits);
                    d = mfma_parts<DT>(k, qf[g * PER + s], d);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const f16x2 sb = keys.steps.at(u, e, g);
                    float mine = own<REP>(d, e, lane);
                    if constexpr (DT == BCONV_BF16) mine = __builtin_fmaf(-24.0f, qsum[g], mine);
                    z[u][e] = __builtin_fmaf((float)sb[0], mine, z[u][e]);
                    z[u][e] = __builtin_fmaf((float)sb[1], qsum[g], z[u][e]);
                }
            }
        }
        // Tiles that some column does not see in full, or with a block that
        // does not exist: masked logits are -inf whatever was read, and masked
        // tokens' steps and midpoints 0, since 0 * NaN would not vanish.
        if (t < all_lo || t + kTokens - 1 > all_hi || !exists(id0) || !exists(id1)) {
            const bool known = lg & 2 ? exists(id1) : exists(id0);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int pos = t + vrun + 4 * u + e * REP + lane % REP;
                    if (!known || pos < lo || pos > hi) z[u][e] = -__builtin_inff();
                }
            values.steps.mask(lane, [&](int i) {
                const int pos = t + vrun + i;
                return known && pos >= sp.low && pos < sp.t1;
            });
        }

        // Running softmax.  The logits are rounded before the maximum is taken
        // off: fused with the subtraction, a logit beyond 2^31 would differ from
        // itself, as the maximum, by more than exp2 holds.
        float p[2][E];
        bool moved = false;  // this column's maximum
        {
#pragma clang fp contract(off)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) z[u][e] *= scale;
            float top = fmaxf(z[0][0], z[1][0]);
#pragma unroll
            for (int e = 1; e < E; ++e) top = fmaxf(top, fmaxf(z[0][e], z[1][e]));
            const uint32_t step = LEAD ? values.steps.top() : 0u;
            // (m + kSlack would round up to a logit that is further away)
            if (__any(top - m > kSlack || step >= limit)) {
                top = fmaxf(m, copies_max<REP>(lane_groups_max(top)));
                float grown = 0.0f;
                if constexpr (LEAD) {
                    uint32_t most = lane_groups_max_bits(step);
#pragma unroll
                    for (int d = 1; d < 16; d *= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d));
                    most = __builtin_amdgcn_readfirstlane(most);
                    if (most >= limit) {
                        limit = ((most >> 10) + 1) << 10;
                        grown = lead_of(limit) - lead;
                        lead += grown;
                    }
                }
                const float f = __builtin_amdgcn_exp2f(m - top + grown);
                moved = top > m;
                m = top;
                l *= f;
#pragma unroll
                for (int k = 0; k < TILES; ++k) acc[k] *= f;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    mid[g] *= f;
                    if constexpr (SUMS) psum[g] *= f;
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    p[u][e] = __builtin_amdgcn_exp2f(LEAD ? z[u][e] - m + lead : z[u][e] - m);
                    l += p[u][e];
                }
        }

        // V^T P; word i of an operand is tokens i and i + 4 of the run
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            if (!FULL && g * VPER * 16 >= a.g.dim) continue;
            float ps[2][E];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const f16x2 sb = values.steps.at(u, e, g);
                    ps[u][e] = __builtin_fmaf((float)sb[0], p[u][e], 0.0f);  // one instruction, with the conversion
                    mid[g] = __builtin_fmaf((float)sb[1], p[u][e], mid[g]);
                }
            if constexpr (UNITS) {
                float top = fmaxf(ps[0][0], ps[1][0]);
#pragma unroll
                for (int e = 1; e < E; ++e) top = fmaxf(top, fmaxf(ps[0][e], ps[1][e]));
                const bool over = top * unit[g] >= 32768.0f;
                if (__any(moved || over)) {
                    top = copies_max<REP>(lane_groups_max(top));
                    // a column keeps its unit unless its own products ask for one
                    if (moved || top * unit[g] >= 32768.0f) {
                        const Unit next(__float_as_uint(top));
                        const float f = next.to * (1.0f / unit[g]);
                        unit[g] = next.to;
#pragma unroll
                        for (int j = 0; j < VPER; ++j) acc[g * VPER + j] *= f;
                    }
                }
            }
            u32x4 pp[NP];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                uint32_t two[NP];
                if constexpr (UNITS) {
                    split_pair(ps[0][e], ps[1][e], unit[g], two[0], two[1]);
                } else if constexpr (LEAD) {
                    const f16x2 r = {(_Float16)ps[0][e], (_Float16)ps[1][e]};
                    two[0] = __builtin_bit_cast(uint32_t, r);
                } else {
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        const bf16x2 r = {(__bf16)ps[0][e], (__bf16)ps[1][e]};
                        two[k] = __builtin_bit_cast(uint32_t, r);
                        ps[0][e] -= (float)r[0];
                        ps[1][e] -= (float)r[1];
                    }
                }
#pragma unroll
                for (int k = 0; k < NP; ++k)
#pragma unroll
                    for (int c = 0; c < REP; ++c) pp[k][e * REP + c] = from_copy<REP>(two[k], c);
            }
            if constexpr (SUMS) psum[g] = mfma16<VT>(offset, pp[0], psum[g]);
#pragma unroll
            for (int j = 0; j < VPER; ++j) {
                const int tile = g * VPER + j, word = tile / 8, half = (tile / 4) & 1;
                u32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = __builtin_amdgcn_perm(values.w[i + 4][word], values.w[i][word],
                                                               half ? 0x07060302u : 0x05040100u);
                    v[i] = value_pair<DT>(two, tile & 3, vbits);
                }
#pragma unroll
                for (int k = NP - 1; k >= 0; --k) {
                    if constexpr (DT != BCONV_F32 && !SUMS) acc[tile] = mfma16<VT>(offset, pp[k], acc[tile]);
                    acc[tile] = mfma16<VT>(v, pp[k], acc[tile]);
                }
            }
        }
    }

    // the waves' sums, brought to one maximum and added in wave order
    extern __shared__ float lds[];
    float *so = lds;                             // [waves][COLS][DP + 4]
    float *sm = lds + WAVES * COLS * (DP + 4);   // [waves][COLS]
    float *sl = sm + WAVES * COLS;
    l = copies_sum<REP>(lane_groups_sum(l));
    if (lg == 0 && row % REP == 0) {
        sm[wave * COLS + col] = m;
        sl[wave * COLS + col] = LEAD ? l * __builtin_amdgcn_exp2f(-lead) : l;
    }
    __syncthreads();
    {
        float top = kLowest;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sm[w * COLS + col]);
        const float f = __builtin_amdgcn_exp2f(m - top - lead);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const float from = UNITS ? 1.0f / unit[g] : 1.0f;  // exact
            float add = copies_sum<REP>(lane_groups_sum(mid[g]));
            if constexpr (SUMS) add -= kValueOffset<DT> * psum[g][0];
#pragma unroll
            for (int j = 0; j < VPER; ++j) {
                const int tile = g * VPER + j;
                if (col < sp.c1 - sp.c0 && row % REP == 0)
                    *reinterpret_cast<f32x4 *>(so + (wave * COLS + col) * (DP + 4) + tile * 16 + lg * 4) =
                        (acc[tile] * from + add) * f;
            }
        }
    }
    __syncthreads();
    const int cols = sp.c1 - sp.c0;
    for (int e = threadIdx.x; e < cols * DP; e += WAVES * 64) {
        const int c = e / DP, d = e % DP;
        if (d >= a.g.dim) continue;
        float top = kLowest, sum = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sm[w * COLS + c]);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            sum += sl[w * COLS + c] * __builtin_amdgcn_exp2f(sm[w * COLS + c] - top);
            o += so[(w * COLS + c) * (DP + 4) + d];
        }
        const int j = (int)fastdiv((uint32_t)(sp.c0 + c), a.by_ratio), h = head * a.ratio + (sp.c0 + c - j * a.ratio);
        const long long at = (long long)(sp.q0 + j) * a.heads + h;
        if (whole) {
            static_cast<T *>(a.out)[at * a.g.dim + d] = round_to<DT>(sum > 0.0f || sum != sum ? o / sum : 0.0f);
            if (a.lse && d == 0) a.lse[at] = sum > 0.0f || sum != sum ? (top + __log2f(sum)) * kLn2 : -__builtin_inff();
        } else {
            a.part_o[(at * a.parts + part) * DP + d] = o;
            if (d == 0) a.part_ml[at * a.parts + part] = float2{top, sum};
        }
    }
}

// Joins the parts of one column, a workgroup each: DP / 4 threads take the
// channels, 2048 / DP slices of them every so-many-th part; the slices are
// added in order.  Bound by its launch and three dependent loads (5 us).
template <int DT, int DP>
__global__ __launch_bounds__(kMaxParts) void kv4_combine_kernel(AttnArgs a)
{
    typedef typename Elem<DT>::type T;
    constexpr int THREADS = DP / 4, SLICES = kMaxParts / THREADS, WAVES = kMaxParts / 64;
    __shared__ float factor[kMaxParts], edge[2 * WAVES];
    __shared__ f32x4 sums[SLICES][THREADS];
    const int per_head = a.max_q * a.ratio;
    const int id = a.first + (int)blockIdx.x, tid = threadIdx.x;
    const int c = id % per_head, head = id / per_head % a.g.kv_heads, req = id / per_head / a.g.kv_heads;
    const Span sp = column_span(a, req, c / kCols);
    const int span = sp.t1 - sp.t0;
    if (c >= sp.c1 || span <= a.part_tokens) return;  // uniform over the workgroup
    const int used = (span + a.part_tokens - 1) / a.part_tokens;
    const int j = (int)fastdiv((uint32_t)c, a.by_ratio), h = head * a.ratio + (c - j * a.ratio);
    const long long at = (long long)(sp.q0 + j) * a.heads + h;
    const float2 mine = tid < used ? a.part_ml[at * a.parts + tid] : float2{kLowest, 0.0f};
    float top = mine.x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    if ((tid & 63) == 0) edge[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) top = fmaxf(top, edge[w]);
    const float f = __builtin_amdgcn_exp2f(mine.x - top);
    factor[tid] = f;
    float sum = mine.y * f;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) edge[WAVES + (tid >> 6)] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += edge[WAVES + w];

    const int d4 = tid % THREADS, slice = tid / THREADS;
    const f32x4 *o4 = reinterpret_cast<const f32x4 *>(a.part_o + at * a.parts * DP) + d4;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
    for (int p = slice; p < used; p += SLICES) o += o4[(long long)p * THREADS] * factor[p];
    sums[slice][d4] = o;
    __syncthreads();
    if (slice) return;
#pragma unroll
    for (int s = 1; s < SLICES; ++s) o += sums[s][d4];
    const bool any = sum > 0.0f || sum != sum;
    if (4 * d4 < a.g.dim) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            static_cast<T *>(a.out)[at * a.g.dim + 4 * d4 + i] = round_to<DT>(any ? o[i] / sum : 0.0f);
    }
    if (a.lse && tid == 0) a.lse[at] = any ? (top + __log2f(sum)) * kLn2 : -__builtin_inff();
}

// ------------------------------------------------------------------ dispatch

template <int DT, int DP, int GROUPS, bool FULL, int REP>
hipError_t launch_attention_full(AttnArgs a, hipStream_t s)
{
    constexpr int WAVES = attn_waves(DT, DP, GROUPS);
    const size_t lds = (size_t)WAVES * (kCols / REP) * (DP + 4 + 2) * sizeof(float);
    const long long grid = (long long)a.requests * a.g.kv_heads * a.col_blocks * a.parts;
    hipError_t e = launch_slices(grid, [&](long long first, unsigned count) {
        a.first = (int)first;
        hipLaunchKernelGGL((kv4_attention_kernel<DT, DP, GROUPS, FULL, REP>), dim3(count), dim3(WAVES * 64), lds, s, a);
    });
    if (e == hipSuccess && a.parts > 1) {
        const long long cols = (long long)a.requests * a.g.kv_heads * a.max_q * a.ratio;
        e = launch_slices(cols, [&](long long first, unsigned count) {
            a.first = (int)first;
            hipLaunchKernelGGL((kv4_combine_kernel<DT, DP>), dim3(count), dim3(kMaxParts), 0, s, a);
        });
    }
    return e;
}

template <int DT, int DP, int GROUPS>
hipError_t launch_attention_kernel(const AttnArgs &a, hipStream_t s)
{
    if (a.g.dim > DP - DP / GROUPS) {
        // 32 requests of up to 8192 tokens, 32 heads over 8: groups of 64 bf16
        // 54.5 us against 58.4, groups of 32 65 against 77, fp32 89 against 105;
        // 777 tokens 7.1 against 7.8.  Two copies of up to eight columns take
        // more registers than they save (64 heads: 72 against 60).
        if (a.max_q * a.ratio <= 4) return launch_attention_full<DT, DP, GROUPS, true, 4>(a, s);
        return launch_attention_full<DT, DP, GROUPS, true, 1>(a, s);
    }
    if constexpr (GROUPS > 1) return launch_attention_full<DT, DP, GROUPS, false, 1>(a, s);
    return hipErrorInvalidValue;  // not reached: one group is never empty
}

template <int DT, int DP>
hipError_t launch_attention_dim(const AttnArgs &a, hipStream_t s)
{
    switch (a.g.groups) {
    case 1: if constexpr (DP <= 128) return launch_attention_kernel<DT, DP, 1>(a, s); else break;
    case 2: return launch_attention_kernel<DT, DP, 2>(a, s);
    case 4: if constexpr (DP >= 128) return launch_attention_kernel<DT, DP, 4>(a, s); else break;
    case 8: if constexpr (DP >= 256) return launch_attention_kernel<DT, DP, 8>(a, s); else break;
    }
    return hipErrorInvalidValue;
}

template <int DT>
hipError_t launch_attention(const AttnArgs &a, hipStream_t s)
{
    switch (a.g.dim_padded) {
    case 64: return launch_attention_dim<DT, 64>(a, s);
    case 128: return launch_attention_dim<DT, 128>(a, s);
    default: return launch_attention_dim<DT, 256>(a, s);
    }
}

}  // namespace bconv

namespace {

using bconv::fail;

struct AttnPlan {
    bconv::AttnArgs a;
    size_t o_bytes, bytes;  // partial results: sums, then (maximum, denominator) pairs
    bool empty;
};

constexpr long long kMaxContext = 1LL << 30;  // tokens of one request

int compute_units()
{
    static thread_local int cached_dev = -1, cached = 0;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 256;
    if (dev != cached_dev) {
        int cus = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) cus = 256;
        cached = cus;
        cached_dev = dev;
    }
    return cached;
}

// Everything that follows from the descriptor and the host arguments; no
// device work.
bconv_status_t plan_attention(const bconv_kv4_desc_t *desc, const bconv_kv4_attention_t *t, AttnPlan *p)
{
    if (!t) return fail(BCONV_ERR_INVALID_ARGUMENT, "args is NULL");
    *p = AttnPlan{};
    bconv::AttnArgs &a = p->a;
    const bconv_status_t st = bconv::kv4_geometry(desc, &a.g);
    if (st != BCONV_OK) return st;
    if (!bconv::dtype_size(t->dtype)) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", t->dtype);
    if (t->requests < 0 || t->q_tokens < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "requests and q_tokens must be >= 0");
    if (t->heads < 1 || t->heads > 65536 || t->heads % a.g.kv_heads)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "heads must be a multiple of kv_heads (%d) up to 65536", a.g.kv_heads);
    p->empty = t->requests == 0 || t->q_tokens == 0;
    if (p->empty) return BCONV_OK;
    if (!t->q_start && t->q_tokens % t->requests)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "without q_start, q_tokens must be a multiple of requests");
    if (t->max_q < 1) return fail(BCONV_ERR_INVALID_ARGUMENT, "max_q must be >= 1");
    if (!t->q_start && t->max_q < t->q_tokens / t->requests)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "max_q is below q_tokens / requests");
    if (t->table_width < 0 || t->table_stride < t->table_width)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "table_width must be >= 0 and table_stride >= table_width");
    if (t->max_context < 0 || t->max_context > kMaxContext || t->window < 0)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "max_context must be in [0, 2^30] and window >= 0");
    if (t->q_token_stride < 0 || t->q_head_stride < 0 || t->q_token_stride > (1LL << 40) || t->q_head_stride > (1LL << 40))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "strides must be in [0, 2^40]");
    const int es = bconv::dtype_size(t->dtype);
    a.pool = static_cast<const char *>(t->pool);
    a.q = t->q;
    a.q_token = t->q_token_stride;
    a.q_head = t->q_head_stride;
    a.out = t->out;
    a.lse = t->lse;
    a.table = t->block_table;
    a.context = t->context_lens;
    a.q_start = t->q_start;
    a.requests = t->requests;
    a.q_tokens = t->q_tokens;
    a.max_q = t->max_q < t->q_tokens ? t->max_q : t->q_tokens;
    a.heads = t->heads;
    a.ratio = t->heads / a.g.kv_heads;
    a.by_ratio = bconv::make_fastdiv((uint32_t)a.ratio);
    a.width = t->table_width;
    a.stride = t->table_stride;
    const long long held = (long long)t->table_width << a.g.block_shift;
    long long most = t->max_context > 0 && t->max_context < held ? t->max_context : held;
    if (most > kMaxContext) most = kMaxContext;
    a.max_context = (int)most;
    a.window = t->window;
    a.scale_log2 = fabsf(t->scale) * bconv::kLog2e;
    a.flip = t->scale < 0.0f ? 0x80008000u : 0u;
    a.vec = (uintptr_t)t->q % 16 == 0 && t->q_token_stride * es % 16 == 0 && t->q_head_stride * es % 16 == 0;

    if ((long long)a.max_q * a.ratio >= (1LL << 30)) return fail(BCONV_ERR_INVALID_ARGUMENT, "max_q*heads too large");
    a.col_blocks = (a.max_q * a.ratio + bconv::kCols - 1) / bconv::kCols;
    const long long tiles = (long long)a.requests * a.g.kv_heads * a.col_blocks;
    if (tiles >= (1LL << 27)) return fail(BCONV_ERR_INVALID_ARGUMENT, "requests*heads*max_q too large for one call");
    // tokens that the columns of one workgroup can see, from a multiple of the tile
    long long seen = most;
    if (a.window > 0) {
        const long long w = (long long)a.window + (bconv::kCols + a.ratio - 1) / a.ratio;
        if (w < seen) seen = w;
    }
    seen += bconv::kTokens;
    // Parts of the long axis: two workgroups a compute unit, a part no shorter
    // than 64 tokens a wave and no more than 128 parts a row, which their join
    // would outweigh, and none longer than 1056 a wave, so that one long request
    // among short ones is shared.  Up to 136 tokens a wave stay whole: the join's
    // launch costs more than the second half of the tokens (777 tokens, two
    // key/value heads: 7.8 us whole, 10.4 in two; 4 requests of 8192 tokens,
    // eight heads: 17 us in parts of 512, 21 in parts of 1024).
    const int waves = bconv::attn_waves(t->dtype, a.g.dim_padded, a.g.groups);
    long long part = seen;
    if (seen > 136 * waves) {
        const long long want = (2LL * compute_units() + tiles - 1) / tiles;
        part = (seen + want - 1) / want;
        if (part < 64 * waves) part = 64 * waves;
        if (part < (seen + 127) / 128) part = (seen + 127) / 128;
        if (part > 1056 * waves && a.col_blocks <= 4) part = 1056 * waves;
        if (part < (seen + bconv::kMaxParts - 1) / bconv::kMaxParts) part = (seen + bconv::kMaxParts - 1) / bconv::kMaxParts;
    }
    part = (part + bconv::kTokens - 1) / bconv::kTokens * bconv::kTokens;
    a.part_tokens = (int)part;
    a.parts = (int)((seen + part - 1) / part);
    if (a.parts < 1) a.parts = 1;
    if (tiles * a.parts >= (1LL << 31)) return fail(BCONV_ERR_INVALID_ARGUMENT, "too many parts for one call");
    if (a.parts > 1) {
        const size_t rows = (size_t)a.q_tokens * a.heads * a.parts;
        p->o_bytes = (rows * a.g.dim_padded * 4 + 255) / 256 * 256;
        p->bytes = p->o_bytes + rows * 8;
    }
    return BCONV_OK;
}

}  // namespace

extern "C" {

bconv_status_t bconv_kv4_attention_workspace_size(const bconv_kv4_desc_t *desc, const bconv_kv4_attention_t *args,
                                                  size_t *bytes)
{
    if (!bytes) return fail(BCONV_ERR_INVALID_ARGUMENT, "bytes is NULL");
    AttnPlan p;
    const bconv_status_t st = plan_attention(desc, args, &p);
    if (st != BCONV_OK) return st;
    *bytes = p.bytes;
    return BCONV_OK;
}

bconv_status_t bconv_kv4_attention(const bconv_kv4_desc_t *desc, void *stream, const bconv_kv4_attention_t *args,
                                   void *workspace, size_t workspace_bytes)
{
    AttnPlan p;
    const bconv_status_t st = plan_attention(desc, args, &p);
    if (st != BCONV_OK) return st;
    if (p.empty) return BCONV_OK;
    if (!args->pool || !args->q || !args->out || !args->context_lens || (!args->block_table && args->table_width > 0))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "pool, q, out, block_table and context_lens must not be NULL");
    const int es = bconv::dtype_size(args->dtype);
    if ((uintptr_t)args->pool % 16 || ((uintptr_t)args->q | (uintptr_t)args->out) % es)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "the pool must be 16-byte aligned, q and out aligned to an element");
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes))
        return fail(BCONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", p.bytes,
                    workspace ? workspace_bytes : (size_t)0);
    if (p.bytes > 0 && (uintptr_t)workspace % 16) return fail(BCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    p.a.part_o = static_cast<float *>(workspace);
    p.a.part_ml = p.bytes ? reinterpret_cast<float2 *>(static_cast<char *>(workspace) + p.o_bytes) : nullptr;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    switch (args->dtype) {
    case BCONV_F32: e = bconv::launch_attention<BCONV_F32>(p.a, s); break;
    case BCONV_F16: e = bconv::launch_attention<BCONV_F16>(p.a, s); break;
    default: e = bconv::launch_attention<BCONV_BF16>(p.a, s); break;
    }
    if (e != hipSuccess) return bconv::hip_fail(e, "cache attention kernel");
    return BCONV_OK;
}

}  // extern "C"
