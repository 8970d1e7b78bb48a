// Tokens to the experts they chose and back: a stable counting sort of the
// (token, choice) pairs, rows into that order, their weighted sums and the
// gradients of both.
#include <hip/hip_runtime.h>

#include "host.h"
#include "mx4.h"

namespace bconv {

// ------------------------------------------------------------------ the sort
//
// A workgroup takes a part of the pairs, its waves a stretch of the part each,
// in order.  Counts by wave and expert are taken in LDS, a scan over experts,
// then waves, turns them into first places, and each wave goes over its stretch again, 64 pairs at
// a time: ballots over the bits of the ids give a lane the lanes with the same
// id, and the number of those before it.  Dropped pairs sort as one more
// expert.  One launch where one workgroup takes all pairs; otherwise one that
// only counts, and one in which every workgroup adds up the counts of those before it.

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxParts = 256;
constexpr int kOnePart = 8192;   // pairs that one workgroup sorts alone
constexpr int kLeastPart = 2048;

struct SortArgs {
    const void *ids;
    int *offsets, *order, *position;
    int *counts;  // [parts][experts + 1]
    int pairs, experts, bits, per_part, parts;
};

template <typename I> __device__ __forceinline__ int key_of(const SortArgs &a, int i)
{
    const I id = static_cast<const I *>(a.ids)[i];
    return id >= 0 && id < (I)a.experts ? (int)id : a.experts;
}

// Pairs [begin, end) of this wave.
__device__ __forceinline__ void stretch(const SortArgs &a, int wave, int &begin, int &end)
{
    const long long first = (long long)blockIdx.x * a.per_part;
    const long long last = first + a.per_part < a.pairs ? first + a.per_part : a.pairs;
    const int each = (a.per_part + kSortThreads - 1) / kSortThreads * 64;
    const long long b = first + (long long)wave * each, e = b + each;
    begin = (int)(b < last ? b : last);
    end = (int)(e < last ? e : last);
}

template <typename I> __device__ __forceinline__ void count_pairs(const SortArgs &a, int *count, int begin, int end, int lane)
{
    for (int i = begin + lane; i < end; i += 64) atomicAdd(&count[key_of<I>(a, i)], 1);  // of this wave alone
}

template <typename I> __global__ __launch_bounds__(kSortThreads) void expert_count_kernel(SortArgs a)
{
    extern __shared__ int count[];  // [experts + 1]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, keys = a.experts + 1;
    for (int e = threadIdx.x; e < keys; e += kSortThreads) count[e] = 0;
    __syncthreads();
    int begin, end;
    stretch(a, wave, begin, end);
    count_pairs<I>(a, count, begin, end, lane);
    __syncthreads();
    for (int e = threadIdx.x; e < keys; e += kSortThreads) a.counts[blockIdx.x * keys + e] = count[e];
}

template <typename I> __global__ __launch_bounds__(kSortThreads) void expert_place_kernel(SortArgs a)
{
    extern __shared__ int count[];  // [waves][experts + 1], counts, then next places
    __shared__ int sums[kSortWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, keys = a.experts + 1;
    for (int e = threadIdx.x; e < keys * kSortWaves; e += kSortThreads) count[e] = 0;
    __syncthreads();
    int begin, end;
    stretch(a, wave, begin, end);
    int *mine = count + wave * keys;
    count_pairs<I>(a, mine, begin, end, lane);
    __syncthreads();
    // a thread has consecutive experts: `total` pairs in all parts, `before` in
    // the parts before this
    constexpr int kEach = (kMaxExperts + 1 + kSortThreads - 1) / kSortThreads;
    const int each = (keys + kSortThreads - 1) / kSortThreads;
    int total[kEach], before[kEach], sum = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = threadIdx.x * each + j;
        total[j] = before[j] = 0;
        if (j >= each || e >= keys) continue;
        if (a.parts == 1) {
            for (int w = 0; w < kSortWaves; ++w) total[j] += count[w * keys + e];
        } else {
#pragma unroll 8
            for (int p = 0; p < a.parts; ++p) {
                const int c = a.counts[p * keys + e];
                total[j] += c;
                before[j] += p < (int)blockIdx.x ? c : 0;
            }
        }
        sum += total[j];
    }
    int upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(upto, d);
        if (lane >= d) upto += u;
    }
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - sum;
    for (int w = 0; w < wave; ++w) at += sums[w];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = threadIdx.x * each + j;
        if (j >= each || e >= keys) continue;
        if (blockIdx.x == 0) a.offsets[e] = at;
        int next = at + before[j];
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = count[w * keys + e];
            count[w * keys + e] = next;
            next += c;
        }
        at += total[j];
    }
    __syncthreads();
    for (int i0 = begin; i0 < end; i0 += 64) {
        const int i = i0 + lane;
        const bool in = i < end;
        const int key = in ? key_of<I>(a, i) : -1;
        unsigned long long same = __ballot(in);
        for (int b = 0; b < a.bits; ++b) {
            const unsigned long long set = __ballot((key >> b) & 1);
            same &= (key >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int p = in ? mine[key] + rank : 0;
        __builtin_amdgcn_wave_barrier();
        if (in && rank == 0) mine[key] = p + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (in) {
            const bool kept = key < a.experts;
            a.order[p] = kept ? i : -1;
            a.position[i] = kept ? p : -1;
        }
    }
}

static int sort_parts(int pairs, int &per_part)
{
    per_part = pairs;
    if (pairs <= kOnePart) return 1;
    per_part = (pairs + kMaxParts - 1) / kMaxParts;
    per_part = (per_part + kSortThreads - 1) / kSortThreads * kSortThreads;
    if (per_part < kLeastPart) per_part = kLeastPart;
    return (pairs + per_part - 1) / per_part;
}

template <typename I> static hipError_t run_sort(const SortArgs &a, hipStream_t s)
{
    const size_t row = (size_t)(a.experts + 1) * sizeof(int);
    if (a.parts > 1) {
        hipLaunchKernelGGL((expert_count_kernel<I>), dim3(a.parts), dim3(kSortThreads), row, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((expert_place_kernel<I>), dim3(a.parts), dim3(kSortThreads), row * kSortWaves, s, a);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the rows

struct RowsArgs {
    const void *from;   // gather: x; combine: rows; backward: rows
    const void *dy;
    const int *order, *position;
    const void *weights;
    void *to;           // gather: rows; combine: y; backward: d_rows
    void *d_weights;
    long long ld_from, ld_dy;
    int tokens, choices, width, pairs;
    int weight_dtype;
    int first;          // token of the launch's first workgroup
};

constexpr int kRowThreads = 256;

template <int DT> constexpr int kPiece = DT == BCONV_F32 ? 4 : 8;  // values of 16 bytes

// What a lane moves at once: 16 bytes of a row, or what is left of it.
template <int DT> struct Piece {
    typedef typename Elem<DT>::type T;
    T v[kPiece<DT>];
    __device__ __forceinline__ static Piece load(const void *base, long long at, int left)
    {
        const T *s = static_cast<const T *>(base) + at;
        if (left >= kPiece<DT>) return __builtin_bit_cast(Piece, (u32x4)*reinterpret_cast<const u32x4_any *>(s));
        Piece p;
#pragma unroll
        for (int i = 0; i < kPiece<DT>; ++i) p.v[i] = i < left ? s[i] : (T)0.0f;
        return p;
    }
    // AWAY: past the caches, which the rows read and written would only fill.
    template <bool AWAY = false> __device__ __forceinline__ void store(void *base, long long at, int left) const
    {
        T *d = static_cast<T *>(base) + at;
        if (left >= kPiece<DT>) {
            u32x4_any *q = reinterpret_cast<u32x4_any *>(d);
            if constexpr (AWAY) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, *this), q);
            else *q = __builtin_bit_cast(u32x4, *this);
            return;
        }
#pragma unroll
        for (int i = 0; i < kPiece<DT>; ++i)
            if (i < left) d[i] = v[i];
    }
};

__device__ __forceinline__ float load_weight(const RowsArgs &a, long long i)
{
    if (!a.weights) return 1.0f;
    if (a.weight_dtype == BCONV_F32) return static_cast<const float *>(a.weights)[i];
    if (a.weight_dtype == BCONV_F16) return (float)static_cast<const _Float16 *>(a.weights)[i];
    return (float)static_cast<const __bf16 *>(a.weights)[i];
}

__device__ __forceinline__ void store_weight(const RowsArgs &a, long long i, float v)
{
    if (a.weight_dtype == BCONV_F32) static_cast<float *>(a.d_weights)[i] = v;
    else if (a.weight_dtype == BCONV_F16) static_cast<_Float16 *>(a.d_weights)[i] = (_Float16)v;
    else static_cast<__bf16 *>(a.d_weights)[i] = (__bf16)v;
}

// The place of a pair, -1 for a dropped one (or one that no sort can have given).
__device__ __forceinline__ int place(const RowsArgs &a, long long pair)
{
    const int p = a.position[pair];
    return p < a.pairs ? p : -1;
}

// Few tokens leave compute units idle: then gridDim.y workgroups share a row.
template <int V> __device__ __forceinline__ int first_value() { return ((int)blockIdx.y * kRowThreads + (int)threadIdx.x) * V; }

// Zeros to the places among those numbered like the token's pairs that are no pair's.
template <int DT> __device__ __forceinline__ void clear_places(const RowsArgs &a, int t)
{
    constexpr int V = kPiece<DT>;
    Piece<DT> zero;
#pragma unroll
    for (int i = 0; i < V; ++i) zero.v[i] = (typename Elem<DT>::type)0.0f;
    for (int j = 0; j < a.choices; ++j) {
        const long long p = (long long)t * a.choices + j;
        if (a.order[p] >= 0) continue;
        for (int c = first_value<V>(); c < a.width; c += gridDim.y * kRowThreads * V) zero.store(a.to, p * a.width + c, a.width - c);
    }
}

constexpr int kFewTokens = 128;  // up to which several workgroups take a token
constexpr int kTogether = 8;  // choices whose rows are in flight at once

// The places of choices j0 .. of a token, -1 for dropped ones and from `end` on.
__device__ __forceinline__ void places(const RowsArgs &a, int t, int j0, int end, int (&at)[kTogether])
{
#pragma unroll
    for (int j = 0; j < kTogether; ++j)
        at[j] = j0 + j < end ? __builtin_amdgcn_readfirstlane(place(a, (long long)t * a.choices + j0 + j)) : -1;
}

// A workgroup a token: its row is read once for kTogether choices and written for
// each.  Bound by its bytes: 8193 tokens of 4096 bf16 values to 4 rows each, 336 MB,
// 52 us (6.4 TB/s; a large copy reaches 4.9, a fill 6.9).
template <int DT, bool AWAY> __global__ __launch_bounds__(kRowThreads) void expert_gather_kernel(RowsArgs a)
{
    constexpr int V = kPiece<DT>;
    const int t = a.first + (int)blockIdx.x;
    for (int j0 = 0; j0 < a.choices; j0 += kTogether) {
        int at[kTogether];
        places(a, t, j0, a.choices, at);
        for (int c = first_value<V>(); c < a.width; c += gridDim.y * kRowThreads * V) {
            const Piece<DT> p = Piece<DT>::load(a.from, t * a.ld_from + c, a.width - c);
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
                if (at[j] >= 0) p.template store<AWAY>(a.to, (long long)at[j] * a.width + c, a.width - c);
        }
    }
    clear_places<DT>(a, t);
}

// A workgroup a token; the rows of kTogether choices are requested before the
// first is added.  MANY: there are more choices than that.  Bound by its bytes:
// the same rows back, 336 MB, 50 us (6.7 TB/s).
template <int DT, bool MANY, bool AWAY> __global__ __launch_bounds__(kRowThreads) void expert_combine_kernel(RowsArgs a)
{
    constexpr int V = kPiece<DT>;
    const int t = a.first + (int)blockIdx.x;
    int at[kTogether];
    float w[kTogether];
    auto choose = [&](int j0) {
        places(a, t, j0, a.choices, at);
#pragma unroll
        for (int j = 0; j < kTogether; ++j) w[j] = at[j] >= 0 ? load_weight(a, (long long)t * a.choices + j0 + j) : 0.0f;
    };
    if constexpr (!MANY) choose(0);
    for (int c = first_value<V>(); c < a.width; c += gridDim.y * kRowThreads * V) {
        float sum[V];
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = 0.0f;
        for (int j0 = 0; j0 < (MANY ? a.choices : 1); j0 += kTogether) {
            if constexpr (MANY) choose(j0);
            Piece<DT> p[kTogether];
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
                if (at[j] >= 0) p[j] = Piece<DT>::load(a.from, at[j] * a.ld_from + c, a.width - c);
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
                if (at[j] >= 0)
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] = __builtin_fmaf(w[j], (float)p[j].v[i], sum[i]);
        }
        Piece<DT> y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.v[i] = (typename Elem<DT>::type)sum[i];
        y.template store<AWAY>(a.to, (long long)t * a.width + c, a.width - c);
    }
}

// A workgroup a token: dy's row is read once for kTogether choices; or, with
// few tokens, one for each choice (gridDim.y of them).  Bound by its bytes: 2049 tokens
// with 6 rows of 5003 fp32 values, 533 MB, 118 us again and again (4.5 TB/s), 135
// with the tokens' gradient between.
template <int DT, bool AWAY> __global__ __launch_bounds__(kRowThreads) void expert_combine_backward_kernel(RowsArgs a)
{
    constexpr int V = kPiece<DT>;
    __shared__ float part[kRowThreads / 64][kTogether];
    const int t = a.first + (int)blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool one = gridDim.y > 1;
    const int end = one ? (int)blockIdx.y + 1 : a.choices;
    for (int j0 = blockIdx.y; j0 < end; j0 += kTogether) {
        int at[kTogether];
        float w[kTogether], dot[kTogether];
        places(a, t, j0, end, at);
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            w[j] = at[j] >= 0 ? load_weight(a, (long long)t * a.choices + j0 + j) : 0.0f;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x * V; c < a.width; c += kRowThreads * V) {
            const int left = a.width - c;
            const Piece<DT> d = Piece<DT>::load(a.dy, t * a.ld_dy + c, left);
            Piece<DT> r[kTogether];
            if (a.d_weights) {
#pragma unroll
                for (int j = 0; j < kTogether; ++j)
                    if (at[j] >= 0) r[j] = Piece<DT>::load(a.from, at[j] * a.ld_from + c, left);
            }
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                if (at[j] < 0) continue;
                Piece<DT> g;
#pragma unroll
                for (int i = 0; i < V; ++i) g.v[i] = (typename Elem<DT>::type)(w[j] * (float)d.v[i]);
                g.template store<AWAY>(a.to, (long long)at[j] * a.width + c, left);
                if (a.d_weights)
#pragma unroll
                    for (int i = 0; i < V; ++i) dot[j] = __builtin_fmaf((float)d.v[i], (float)r[j].v[i], dot[j]);
            }
        }
        if (a.d_weights) {
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                if (j0 + j >= end) break;
#pragma unroll
                for (int d = 32; d > 0; d /= 2) dot[j] += __shfl_xor(dot[j], d);
                if (lane == 0) part[wave][j] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < kTogether && j0 + (int)threadIdx.x < end) {
                float sum = part[0][threadIdx.x];
                for (int v = 1; v < kRowThreads / 64; ++v) sum += part[v][threadIdx.x];
                store_weight(a, (long long)t * a.choices + j0 + threadIdx.x, sum);
            }
            __syncthreads();
        }
    }
    clear_places<DT>(a, t);
}

enum RowsOp { kGather, kCombine, kCombineBackward };

template <int DT, bool AWAY> static void launch_rows(RowsOp op, const RowsArgs &a, dim3 grid, hipStream_t s)
{
    switch (op) {
    case kGather: hipLaunchKernelGGL((expert_gather_kernel<DT, AWAY>), grid, dim3(kRowThreads), 0, s, a); break;
    case kCombine:
        if (a.choices > kTogether) hipLaunchKernelGGL((expert_combine_kernel<DT, true, AWAY>), grid, dim3(kRowThreads), 0, s, a);
        else hipLaunchKernelGGL((expert_combine_kernel<DT, false, AWAY>), grid, dim3(kRowThreads), 0, s, a);
        break;
    default: hipLaunchKernelGGL((expert_combine_backward_kernel<DT, AWAY>), grid, dim3(kRowThreads), 0, s, a);
    }
}

template <int DT> static hipError_t run_rows(RowsOp op, RowsArgs a, hipStream_t s)
{
    // Through the caches and past them: 32772 rows of 4096 bf16 values gathered 67.5 us, 52.4; combined 64.4, 51.6;
    // gradients 146, 140; 12294 rows of 5003 fp32 values combined 45.3, 44.7, gradients 134, 118; 16392 of 4096
    // bf16 gradients 72, 53.  The next kernel pays part of it: with one that reads the result, gathered 156, 159,
    // combined (and added to as many rows) 97, 103, gradients and the tokens' 213, 203; 190, 191; 101, 98.
    // 8200 rows of 4096 (64 MiB): 15.1, 18.2; 15.2, 15.1; 29.3, 28.9, with the next 37, 41; 20.4, 20.5; 43, 46.
    // A combination goes by the rows that it reads, not the fewer that it stores: 41 MB of 246 between gradients, the pass of
    // both 193, 191; 16 MB of 134 alone 28.1, 28.3, with a kernel that reads them 36.7, 37.7.
    // Gathered rows that end inside a line are better put together in the caches (5003 fp32 values: 66, 73).
    const int es = DT == BCONV_F32 ? 4 : 2;
    const bool away = (long long)a.pairs * a.width * es > 1LL << 26 && (op != kGather || a.width * es % 128 == 0);
    // 64 tokens of 8 rows of 7168 bf16 values: gradients 15.2 us, 10.1 shared, combined 8.7, 7.6; 256 of 4096: 11.4, 13.7.
    const int pieces = (a.width + kRowThreads * kPiece<DT> - 1) / (kRowThreads * kPiece<DT>);
    const unsigned share = a.tokens > kFewTokens ? 1 : op == kCombineBackward ? (unsigned)a.choices : (unsigned)pieces;
    return launch_slices(a.tokens, [&](long long first, unsigned groups) {
        a.first = (int)first;
        const dim3 grid(groups, share < 1024 ? share : op == kCombineBackward ? 1 : 1024);
        if (away) launch_rows<DT, true>(op, a, grid, s);
        else launch_rows<DT, false>(op, a, grid, s);
    });
}

}  // namespace bconv

namespace {

using bconv::fail;
using bconv::hip_fail;
using bconv::kMaxPairs;
using bconv::ranges_overlap;

int bytes_of(int32_t dtype)
{
    return dtype == BCONV_F32 ? 4 : dtype == BCONV_F16 || dtype == BCONV_BF16 ? 2 : 0;
}

bconv_status_t check_sort(int32_t pairs, int32_t experts)
{
    if (pairs < 0 || pairs > kMaxPairs) return fail(BCONV_ERR_INVALID_ARGUMENT, "pairs must be in [0, 2^27]");
    if (experts < 1 || experts > bconv::kMaxExperts)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "experts must be in [1, %d]", bconv::kMaxExperts);
    return BCONV_OK;
}

struct Buffer {
    const void *p;
    size_t n;
};

template <int N, int M> bool any_overlap(const Buffer (&in)[N], const Buffer (&out)[M])
{
    for (int o = 0; o < M; ++o) {
        if (!out[o].p || !out[o].n) continue;
        for (int i = 0; i < N; ++i)
            if (in[i].p && in[i].n && ranges_overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return true;
        for (int i = 0; i < o; ++i)
            if (out[i].p && out[i].n && ranges_overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return true;
    }
    return false;
}

bconv_status_t check_rows(int32_t tokens, int32_t choices, int32_t width, int32_t dtype, int64_t ld, const char *name)
{
    if (!bytes_of(dtype)) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown dtype %d", dtype);
    if (tokens < 0 || choices < 1 || (long long)tokens * choices > kMaxPairs)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "tokens >= 0, choices >= 1 and tokens*choices <= 2^27 are needed");
    if (width < 1 || width > (1 << 20)) return fail(BCONV_ERR_INVALID_ARGUMENT, "width must be in [1, %d]", 1 << 20);
    if (ld < width || ld > bconv::kMaxStride) return fail(BCONV_ERR_INVALID_ARGUMENT, "%s must be in [width, 2^30]", name);
    return BCONV_OK;
}

bconv_status_t finish(bconv::RowsOp op, const bconv::RowsArgs &a, int32_t dtype, void *stream)
{
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e;
    switch (dtype) {
    case BCONV_F32: e = bconv::run_rows<BCONV_F32>(op, a, s); break;
    case BCONV_F16: e = bconv::run_rows<BCONV_F16>(op, a, s); break;
    default: e = bconv::run_rows<BCONV_BF16>(op, a, s); break;
    }
    if (e != hipSuccess) return hip_fail(e, "expert rows kernel");
    return BCONV_OK;
}

}  // namespace

extern "C" {

bconv_status_t bconv_expert_sort_workspace_size(int32_t pairs, int32_t experts, size_t *bytes)
{
    const bconv_status_t st = check_sort(pairs, experts);
    if (st != BCONV_OK) return st;
    if (!bytes) return fail(BCONV_ERR_INVALID_ARGUMENT, "bytes is NULL");
    int per_part;
    const int parts = bconv::sort_parts(pairs, per_part);
    *bytes = parts > 1 ? (size_t)parts * (experts + 1) * sizeof(int) : 0;
    return BCONV_OK;
}

bconv_status_t bconv_expert_sort(void *stream, int32_t pairs, int32_t experts, int32_t id_bytes, const void *ids,
                                 int32_t *offsets, int32_t *order, int32_t *position, void *workspace, size_t workspace_bytes)
{
    const bconv_status_t st = check_sort(pairs, experts);
    if (st != BCONV_OK) return st;
    if (id_bytes != 4 && id_bytes != 8) return fail(BCONV_ERR_INVALID_ARGUMENT, "id_bytes must be 4 or 8");
    if (!offsets || (pairs > 0 && (!ids || !order || !position)))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "ids, offsets, order and position must not be NULL");
    if ((uintptr_t)ids % id_bytes || ((uintptr_t)offsets | (uintptr_t)order | (uintptr_t)position) % 4)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "ids, offsets, order or position not aligned to an element");
    bconv::SortArgs a{};
    a.parts = bconv::sort_parts(pairs, a.per_part);
    const size_t need = a.parts > 1 ? (size_t)a.parts * (experts + 1) * sizeof(int) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(BCONV_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? workspace_bytes : (size_t)0);
    if (need && (uintptr_t)workspace % 16) return fail(BCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    const Buffer in[] = {{ids, (size_t)pairs * id_bytes}};
    const Buffer out[] = {{offsets, ((size_t)experts + 1) * 4}, {order, (size_t)pairs * 4}, {position, (size_t)pairs * 4}, {workspace, need}};
    if (any_overlap(in, out)) return fail(BCONV_ERR_INVALID_ARGUMENT, "results and workspace must overlap neither ids nor each other");
    a.ids = ids;
    a.offsets = offsets;
    a.order = order;
    a.position = position;
    a.counts = static_cast<int *>(workspace);
    a.pairs = pairs;
    a.experts = experts;
    while ((1 << a.bits) <= experts) ++a.bits;  // keys 0 .. experts
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = id_bytes == 4 ? bconv::run_sort<int32_t>(a, s) : bconv::run_sort<int64_t>(a, s);
    if (e != hipSuccess) return hip_fail(e, "expert sort kernel");
    return BCONV_OK;
}

bconv_status_t bconv_expert_gather(void *stream, int32_t tokens, int32_t choices, int32_t width, int32_t dtype, const void *x,
                                   int64_t ldx, const int32_t *order, const int32_t *position, void *rows)
{
    const bconv_status_t st = check_rows(tokens, choices, width, dtype, ldx, "ldx");
    if (st != BCONV_OK) return st;
    if (tokens == 0) return BCONV_OK;
    if (!x || !order || !position || !rows) return fail(BCONV_ERR_INVALID_ARGUMENT, "x, order, position and rows must not be NULL");
    const int es = bytes_of(dtype);
    if (((uintptr_t)x | (uintptr_t)rows) % es || ((uintptr_t)order | (uintptr_t)position) % 4)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "a buffer is not aligned to an element");
    const size_t pairs = (size_t)tokens * choices;
    const Buffer in[] = {{x, ((size_t)(tokens - 1) * ldx + width) * es}, {order, pairs * 4}, {position, pairs * 4}};
    const Buffer out[] = {{rows, pairs * width * es}};
    if (any_overlap(in, out)) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows overlaps x, order or position");
    bconv::RowsArgs a{};
    a.from = x;
    a.ld_from = ldx;
    a.order = order;
    a.position = position;
    a.to = rows;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.pairs = (int)pairs;
    return finish(bconv::kGather, a, dtype, stream);
}

bconv_status_t bconv_expert_combine(void *stream, int32_t tokens, int32_t choices, int32_t width, int32_t dtype, const void *rows,
                                    int64_t ldr, const int32_t *position, int32_t weight_dtype, const void *weights, void *y)
{
    const bconv_status_t st = check_rows(tokens, choices, width, dtype, ldr, "ldr");
    if (st != BCONV_OK) return st;
    const int es = bytes_of(dtype), ws = bytes_of(weight_dtype);
    if (weights && !ws) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown weight_dtype %d", weight_dtype);
    if (tokens == 0) return BCONV_OK;
    if (!rows || !position || !y) return fail(BCONV_ERR_INVALID_ARGUMENT, "rows, position and y must not be NULL");
    if (((uintptr_t)rows | (uintptr_t)y) % es || (uintptr_t)position % 4 || (weights && (uintptr_t)weights % ws))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "a buffer is not aligned to an element");
    const size_t pairs = (size_t)tokens * choices;
    const Buffer in[] = {{rows, ((pairs - 1) * ldr + width) * es}, {position, pairs * 4}, {weights, pairs * ws}};
    const Buffer out[] = {{y, (size_t)tokens * width * es}};
    if (any_overlap(in, out)) return fail(BCONV_ERR_INVALID_ARGUMENT, "y overlaps rows, position or weights");
    bconv::RowsArgs a{};
    a.from = rows;
    a.ld_from = ldr;
    a.position = position;
    a.weights = weights;
    a.weight_dtype = weight_dtype;
    a.to = y;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.pairs = (int)pairs;
    return finish(bconv::kCombine, a, dtype, stream);
}

bconv_status_t bconv_expert_combine_backward(void *stream, int32_t tokens, int32_t choices, int32_t width, int32_t dtype,
                                             const void *dy, int64_t ldd, const void *rows, int64_t ldr, const int32_t *order,
                                             const int32_t *position, int32_t weight_dtype, const void *weights, void *d_rows,
                                             void *d_weights)
{
    bconv_status_t st = check_rows(tokens, choices, width, dtype, ldd, "ldd");
    if (st == BCONV_OK && d_weights) st = check_rows(tokens, choices, width, dtype, ldr, "ldr");
    if (st != BCONV_OK) return st;
    const int es = bytes_of(dtype), ws = bytes_of(weight_dtype);
    if ((weights || d_weights) && !ws) return fail(BCONV_ERR_INVALID_ARGUMENT, "unknown weight_dtype %d", weight_dtype);
    if (tokens == 0) return BCONV_OK;
    if (!dy || !order || !position || !d_rows || (d_weights && !rows))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "dy, order, position, d_rows (and rows for d_weights) must not be NULL");
    if (((uintptr_t)dy | (uintptr_t)d_rows | (d_weights ? (uintptr_t)rows : 0)) % es || ((uintptr_t)order | (uintptr_t)position) % 4 ||
        ((weights || d_weights) && ((uintptr_t)weights | (uintptr_t)d_weights) % ws))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "a buffer is not aligned to an element");
    const size_t pairs = (size_t)tokens * choices;
    const Buffer in[] = {{dy, ((size_t)(tokens - 1) * ldd + width) * es}, {rows, d_weights ? ((pairs - 1) * ldr + width) * es : 0},
                         {order, pairs * 4}, {position, pairs * 4}, {weights, pairs * ws}};
    const Buffer out[] = {{d_rows, pairs * width * es}, {d_weights, pairs * ws}};
    if (any_overlap(in, out))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "d_rows and d_weights must overlap neither an input nor each other");
    bconv::RowsArgs a{};
    a.from = rows;
    a.ld_from = ldr;
    a.dy = dy;
    a.ld_dy = ldd;
    a.order = order;
    a.position = position;
    a.weights = weights;
    a.weight_dtype = weight_dtype;
    a.to = d_rows;
    a.d_weights = d_weights;
    a.tokens = tokens;
    a.choices = choices;
    a.width = width;
    a.pairs = (int)pairs;
    return finish(bconv::kCombineBackward, a, dtype, stream);
}

}  // extern "C"
