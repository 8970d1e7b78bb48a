// Block tables and slot maps of a paged cache from request lengths, in one
// launch.
//
// Two prefix sums over the requests (new tokens, new blocks) place everything:
// new token i of request r has position context[r] + i, and its block is an
// old entry of the table row or free block first[r] + (entry - have[r]).  Every
// workgroup forms both sums for itself in LDS (a few thousand integers at
// most), which costs less than a second launch or a grid-wide wait, then takes
// its share of the tokens and finds a token's request by bisection.  An entry e
// that a request gains starts at position e * block_size, which is always one
// of its new tokens: that token's thread writes the entry, so no thread reads
// what another writes.
//
// Bound by its launch and the chain of loads, sums and a bisection: 2.9 us for
// one token of 32 requests, 5.2 us for 45,000 tokens of 300 requests.
#include <hip/hip_runtime.h>

#include "host.h"
#include "bconv_q4.h"

namespace bconv {

constexpr int kTableThreads = 256;
constexpr int kMaxRequests = 8192;

struct TableArgs {
    int requests, shift, width;
    long long stride;
    int *table;
    const int *context, *added, *free_blocks, *free_head;
    int free_count, tokens;
    int *free_head_out, *slots, *positions, *q_start, *context_out;
};

__device__ __forceinline__ long long clamp_length(int v) { return v < 0 ? 0 : v; }

__device__ __forceinline__ int to_int(long long v) { return v > 0x7fffffffLL ? 0x7fffffff : (int)v; }

// Blocks a request has, and gains.
__device__ __forceinline__ void blocks_of(const TableArgs &a, long long ctx, long long add, long long &have, long long &gain)
{
    const long long round = (1LL << a.shift) - 1;
    have = (ctx + round) >> a.shift;
    long long need = (ctx + add + round) >> a.shift;
    if (need > a.width) need = a.width;
    gain = need > have ? need - have : 0;
}

__global__ __launch_bounds__(kTableThreads) void block_tables_kernel(TableArgs a)
{
    extern __shared__ int lds[];
    int *start = lds;                    // [requests + 1] first new token
    int *first = lds + a.requests + 1;   // [requests] first free block, from *free_head
    __shared__ long long sum_t[kTableThreads / 64], sum_b[kTableThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.requests + kTableThreads - 1) / kTableThreads;
    const int r0 = min(tid * per, a.requests), r1 = min(r0 + per, a.requests);

    long long t = 0, b = 0;
    for (int r = r0; r < r1; ++r) {
        const long long add = clamp_length(a.added[r]);
        long long have, gain;
        blocks_of(a, clamp_length(a.context[r]), add, have, gain);
        t += add;
        b += gain;
    }
    long long it = t, ib = b;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const long long ut = __shfl_up(it, d), ub = __shfl_up(ib, d);
        if (lane >= d) {
            it += ut;
            ib += ub;
        }
    }
    if (lane == 63) {
        sum_t[wave] = it;
        sum_b[wave] = ib;
    }
    __syncthreads();
    long long bt = 0, bb = 0, all_t = 0, all_b = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 64; ++w) {
        if (w < wave) {
            bt += sum_t[w];
            bb += sum_b[w];
        }
        all_t += sum_t[w];
        all_b += sum_b[w];
    }
    bt += it - t;
    bb += ib - b;
    const int head = *a.free_head;
    const bool lead = blockIdx.x == 0;
    for (int r = r0; r < r1; ++r) {
        const long long ctx = clamp_length(a.context[r]), add = clamp_length(a.added[r]);
        long long have, gain;
        blocks_of(a, ctx, add, have, gain);
        start[r] = to_int(bt);
        first[r] = to_int(bb);
        if (lead) {
            if (a.q_start) a.q_start[r] = to_int(bt);
            if (a.context_out) a.context_out[r] = to_int(ctx + add);
        }
        bt += add;
        bb += gain;
    }
    const int total = to_int(all_t);
    if (tid == 0) {
        start[a.requests] = total;
        if (lead) {
            if (a.q_start) a.q_start[a.requests] = total;
            *a.free_head_out = to_int(head + all_b);
        }
    }
    __syncthreads();

    const long long end = total > a.tokens ? total : a.tokens;
    const long long step = (long long)gridDim.x * kTableThreads;
    for (long long i = (long long)blockIdx.x * kTableThreads + tid; i < end; i += step) {
        int slot = -1, pos = 0;
        if (i < total) {
            int lo = 0, hi = a.requests;  // start[lo] <= i < start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= i) lo = mid;
                else hi = mid;
            }
            const long long ctx = clamp_length(a.context[lo]), p = ctx + (i - start[lo]);
            const long long have = (ctx + (1LL << a.shift) - 1) >> a.shift, entry = p >> a.shift;
            const int off = (int)(p & ((1LL << a.shift) - 1));
            pos = to_int(p);
            if (entry < a.width) {
                int block;
                int *cell = a.table + lo * a.stride + entry;
                if (entry < have) {
                    block = *cell;
                } else {
                    const long long f = (long long)head + first[lo] + (entry - have);
                    block = f >= 0 && f < a.free_count ? a.free_blocks[f] : -1;
                    if (off == 0) *cell = block;
                }
                if (block >= 0) slot = (int)(((unsigned)block << a.shift) + (unsigned)off);
            }
        }
        if (i < a.tokens) {
            if (a.slots) a.slots[i] = slot;
            if (a.positions) a.positions[i] = pos;
        }
    }
}

}  // namespace bconv

using bconv::fail;

extern "C" bconv_status_t bconv_block_tables(void *stream, int32_t requests, int32_t block_size, int32_t *block_table,
                                             int32_t table_width, int32_t table_stride, const int32_t *context_lens,
                                             const int32_t *new_lens, const int32_t *free_blocks, int32_t free_count,
                                             const int32_t *free_head, int32_t *free_head_out, int32_t tokens,
                                             int32_t *slots, int32_t *positions, int32_t *q_start,
                                             int32_t *context_lens_out)
{
    if (requests < 0 || requests > bconv::kMaxRequests)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "requests must be in [0, %d]", bconv::kMaxRequests);
    if (block_size < 16 || block_size > 1024 || (block_size & (block_size - 1)))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "block_size must be a power of two in [16, 1024]");
    if (table_width < 0 || table_stride < table_width)
        return fail(BCONV_ERR_INVALID_ARGUMENT, "table_width must be >= 0 and table_stride >= table_width");
    if (free_count < 0 || tokens < 0) return fail(BCONV_ERR_INVALID_ARGUMENT, "free_count and tokens must be >= 0");
    if (!free_head || !free_head_out) return fail(BCONV_ERR_INVALID_ARGUMENT, "free_head/free_head_out is NULL");
    if (requests > 0 && (!context_lens || !new_lens || (table_width > 0 && !block_table)))
        return fail(BCONV_ERR_INVALID_ARGUMENT, "block_table, context_lens and new_lens must not be NULL");
    if (free_count > 0 && !free_blocks) return fail(BCONV_ERR_INVALID_ARGUMENT, "free_blocks is NULL");
    // every workgroup reads the inputs while the first writes results
    const struct { const int32_t *p; size_t n; } in[] = {
        {context_lens, (size_t)requests}, {new_lens, (size_t)requests}, {free_blocks, (size_t)free_count}, {free_head, 1},
        {block_table, requests && table_width ? (size_t)(requests - 1) * table_stride + table_width : 0}},
        out[] = {{context_lens_out, (size_t)requests}, {q_start, (size_t)requests + 1}, {slots, (size_t)tokens},
                 {positions, (size_t)tokens}, {free_head_out, 1}};
    for (const auto &o : out)
        for (const auto &i : in)
            if (o.p && i.p && o.n && i.n && bconv::ranges_overlap(i.p, i.n * 4, o.p, o.n * 4))
                return fail(BCONV_ERR_INVALID_ARGUMENT, "a result overlaps block_table, a length, free_blocks or free_head");
    bconv::TableArgs a{};
    a.requests = requests;
    a.shift = __builtin_ctz((unsigned)block_size);
    a.width = table_width;
    a.stride = table_stride;
    a.table = block_table;
    a.context = context_lens;
    a.added = new_lens;
    a.free_blocks = free_blocks;
    a.free_head = free_head;
    a.free_count = free_count;
    a.tokens = tokens;
    a.free_head_out = free_head_out;
    a.slots = slots;
    a.positions = positions;
    a.q_start = q_start;
    a.context_out = context_lens_out;
    // one workgroup covers a decoding step; prompts get one a 256 tokens, up to two a compute unit
    const int want = (tokens + bconv::kTableThreads - 1) / bconv::kTableThreads;
    const int grid = want < 1 ? 1 : want > 512 ? 512 : want;
    const size_t lds = ((size_t)2 * requests + 1) * sizeof(int);
    hipLaunchKernelGGL(bconv::block_tables_kernel, dim3(grid), dim3(bconv::kTableThreads), lds,
                       static_cast<hipStream_t>(stream), a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return bconv::hip_fail(e, "block table kernel");
    return BCONV_OK;
}
