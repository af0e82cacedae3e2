// Page tables of the key/value cache kept on the GPU: the pages and slots of a
// step's new tokens from the sequences' lengths, and the way back.
//
// "ROCm: enable trillion-parameter MoE models with INT4-FP8 single node",
// config.json (kv_cache_scheme): the cache whose pages these are. The pages have no
// counterpart for the tables themselves, which a serving program there keeps on the host.
//
// Free pages stand on a stack. Sequence b, with len_b tokens and add_b new ones,
// needs n_b = ceil((len_b + add_b) / page) - ceil(len_b / page) pages; in the order
// of b they are taken off the top, so the j-th page taken is stack[count - 1 - j]
// and everything follows from two prefix sums over the sequences. Every block adds
// these up for itself (4096 sequences: 16 values a thread), then the blocks share
// the tokens and the new table entries between them; who a token or a page belongs
// to is found by bisection. Nothing that one block writes does another one read but
// the lengths and the count, which the last block to have read them writes (and, where a
// table is broken, the pages given back, which that block writes once more).
//
// Bound by latency: lengths, sums, page, slot one after another. 256 sequences' step
// takes 3.7 us, and as much to take back; 1024 sequences with 102912 tokens 7.4 and 3.8 us.
#include "internal.h"
#include "kv8.cuh"
#include "pages.cuh"
#include "ptx.cuh"

namespace w4a8 {

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;   // tokens of a thread

// The last i of [0, n) with sums[i] <= x (sums rises from 0 and n >= 1).
__device__ __forceinline__ int owner(const int* sums, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// What stands before each thread of the block: exclusive prefix sums of two values,
// which stop growing at their limits (sums of natural numbers cut off that way
// still associate).
__device__ __forceinline__ void block_before(unsigned& x, unsigned& y, unsigned most_x, unsigned most_y)
{
    __shared__ unsigned sx[kThreads / 32], sy[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned dx = __shfl_up_sync(0xFFFFFFFFu, x, o), dy = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) {
            x = min(x + dx, most_x);
            y = min(y + dy, most_y);
        }
    }
    if (lane == 31)
        sx[warp] = x, sy[warp] = y;
    __syncthreads();
    x = __shfl_up_sync(0xFFFFFFFFu, x, 1);
    y = __shfl_up_sync(0xFFFFFFFFu, y, 1);
    if (lane == 0)
        x = y = 0;
    for (int w = 0; w < warp; ++w) {
        x = min(x + sx[w], most_x);
        y = min(y + sy[w], most_y);
    }
}

__device__ __forceinline__ int pages_of(int tokens, int shift)   // tokens >= 0
{
    return static_cast<int>((static_cast<unsigned>(tokens) + (1u << shift) - 1) >> shift);
}
// The pages on the stack, read by one thread for the block (a barrier has to follow).
__device__ __forceinline__ void read_count(const PagePool& p, int* count)
{
    if (threadIdx.x == 0) {
        const int n = *p.count;
        if (n < 0 || n > p.num_pages)
            set_error(p.err, kErrBitIndex);
        *count = min(max(n, 0), p.num_pages);
    }
}
// Whether this block is the last of the grid to come here; all threads agree. What
// the others have read into shared memory before, they have read. `flag`, which the
// block's threads may have raised before, is in the last block whether any block's was.
__device__ __forceinline__ bool last_block(uint32_t* ticket, int* flag)
{
    __shared__ bool last;
    __syncthreads();
    if (gridDim.x == 1)
        return true;
    if (threadIdx.x == 0) {
        __threadfence();
        const uint32_t seen = atomicAdd(ticket, *flag ? 0x10001u : 1u);   // blocks, and above them those with the flag
        last = (seen & 0xFFFFu) == gridDim.x - 1;
        if (last) {
            *ticket = 0;
            *flag |= seen >> 16;
        }
        __threadfence();
    }
    __syncthreads();
    return last;
}

}  // namespace

__global__ void __launch_bounds__(kThreads) pages_extend_kernel(const __grid_constant__ PagesExtend a)
{
    extern __shared__ int smem[];
    int* starts = smem;               // [B + 1] tokens before each sequence, T + 1 at most
    int* ahead = smem + a.B + 1;      // [B + 1] pages that those before it need, num_pages + 1 at most
    int* have = ahead + a.B + 1;      // [B] its tokens; less than 0 (the complement) where it gets no pages
    __shared__ int taken, count, none;
    const int tid = threadIdx.x, shift = a.p.page_shift;
    if (tid == 0)
        taken = none = 0;
    grid_dep_wait();
    read_count(a.p, &count);
    const int64_t most_tokens = static_cast<int64_t>(a.p.max_pages) << shift;

    // ---- the sums: a thread takes `per` sequences in a row
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    const unsigned most_x = static_cast<unsigned>(a.T) + 1, most_y = static_cast<unsigned>(a.p.num_pages) + 1;
    unsigned x = 0, y = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const int len = a.lens[b], add = max(a.add[b], 0);
        const bool ok = len >= 0 && a.add[b] >= 0 && static_cast<int64_t>(len) + add <= most_tokens;
        bad |= !ok;
        have[b] = ok ? len : ~max(len, 0);
        starts[b + 1] = add;
        ahead[b + 1] = ok ? pages_of(len + add, shift) - pages_of(len, shift) : 0;
        x = min(x + add, most_x);
        y = min(y + ahead[b + 1], most_y);
    }
    block_before(x, y, most_x, most_y);
    if (tid == 0)
        starts[0] = 0, ahead[0] = 0;
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int need = ahead[b + 1];
        x = min(x + static_cast<unsigned>(starts[b + 1]), most_x);
        y = min(y + static_cast<unsigned>(need), most_y);
        starts[b + 1] = static_cast<int>(x);
        ahead[b + 1] = static_cast<int>(y);
        const bool room = x <= static_cast<unsigned>(a.T), there = need == 0 || y <= static_cast<unsigned>(count);
        if (!room && blockIdx.x == 0)
            bad = true;
        if (!there && blockIdx.x == 0)
            set_error(a.p.err, kErrBitPages);
        if (!(room && there) && have[b] >= 0)
            have[b] = ~have[b];
        if (need && have[b] >= 0)
            mine = static_cast<int>(y);
    }
    if (bad && blockIdx.x == 0)
        set_error(a.p.err, kErrBitIndex);
    if (mine)
        atomicMax(&taken, mine);   // those that get pages are the first of those that need some
    const bool last = last_block(a.p.ticket, &none);

    if (blockIdx.x == 0)
        for (int b = tid; b <= a.B; b += kThreads)
            a.starts[b] = min(starts[b], a.T);
    // ---- the new entries of the tables
    const int step = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
    for (int j = first; j < taken; j += step) {
        const int b = owner(ahead, a.B, j);
        const int64_t at = pages_of(have[b], shift) + j - ahead[b];
        a.p.table[b * a.p.stride + at] = a.p.stack[count - 1 - j];
    }
    // ---- the tokens
    const int total = min(starts[a.B], a.T);
    for (int t = first; t < a.T; t += step) {
        int seq = -1, pos = 0, seen = 0, slot = -1;
        if (t < total) {
            seq = owner(starts, a.B, t);
            const int len = have[seq];
            pos = static_cast<int>(static_cast<unsigned>(len < 0 ? ~len : len) + static_cast<unsigned>(t - starts[seq]));
            seen = len < 0 ? 0 : pos + 1;
            if (len >= 0) {
                const int at = pos >> shift, used = pages_of(len, shift);
                const int page = at < used ? a.p.table[seq * a.p.stride + at]
                                           : a.p.stack[count - 1 - (ahead[seq] + at - used)];
                if (static_cast<unsigned>(page) < static_cast<unsigned>(a.p.num_pages))
                    slot = (page << shift) + (pos & ((1 << shift) - 1));
                else
                    set_error(a.p.err, kErrBitIndex);
            }
        }
        a.seqs[t] = seq;
        a.positions[t] = pos;
        a.seen[t] = seen;
        a.slots[t] = slot;
    }
    if (last) {   // every block has read the lengths and the count
        for (int b = tid; b < a.B; b += kThreads) {
            const int len = have[b];
            a.lens_out[b] = len >= 0 ? len + (starts[b + 1] - starts[b]) : a.lens[b];
        }
        if (tid == 0)
            *a.p.count = count - taken;
    }
}

__global__ void __launch_bounds__(kThreads) pages_truncate_kernel(const __grid_constant__ PagesTruncate a)
{
    extern __shared__ int smem[];
    int* ahead = smem;             // [B + 1] pages that those before it give back, num_pages + 1 at most
    int* kept = smem + a.B + 1;    // [B] tokens
    __shared__ int count, broken;  // broken: a page number out of range was met
    const int tid = threadIdx.x, shift = a.p.page_shift;
    if (tid == 0)
        broken = 0;
    grid_dep_wait();
    read_count(a.p, &count);
    const int64_t most_tokens = static_cast<int64_t>(a.p.max_pages) << shift;
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    const unsigned most = static_cast<unsigned>(a.p.num_pages) + 1;
    unsigned x = 0, unused = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const int len = a.lens[b], keep = a.keep[b];
        const bool ok = keep >= 0 && keep <= len && len <= most_tokens;
        bad |= !ok;
        kept[b] = ok ? keep : len;
        ahead[b + 1] = ok ? pages_of(len, shift) - pages_of(keep, shift) : 0;
        x = min(x + ahead[b + 1], most);
    }
    block_before(x, unused, most, most);
    if (tid == 0)
        ahead[0] = 0;
    for (int b = b0; b < b1; ++b) {
        x = min(x + static_cast<unsigned>(ahead[b + 1]), most);
        ahead[b + 1] = static_cast<int>(x);
    }
    __syncthreads();
    // more pages than the stack has room for: somebody's length is wrong, and nothing goes back
    int given = ahead[a.B];
    bool fits = given <= a.p.num_pages - count;
    if ((bad || !fits) && blockIdx.x == 0)
        set_error(a.p.err, kErrBitIndex);
    if (fits) {
        for (int j = blockIdx.x * kThreads + tid; j < given; j += gridDim.x * kThreads) {
            const int b = owner(ahead, a.B, j);
            const int64_t at = pages_of(kept[b], shift) + j - ahead[b];
            const int page = a.p.table[b * a.p.stride + at];
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.p.num_pages)) {
                set_error(a.p.err, kErrBitIndex);
                broken = 1;
            }
            // in reverse: what an extension took comes to lie as it lay
            a.p.stack[count + given - 1 - j] = page;
        }
    }
    // the last block to have done its part writes the lengths and the count, which all have read
    if (!last_block(a.p.ticket, &broken))
        return;
    if (broken || !fits) {
        // Sequences with a page number out of range among those to go keep all, so that no
        // such number comes to the stack; the others' pages are written again, by this block.
        for (int b = 0; b < a.B; ++b) {
            const int len = a.lens[b], end = kept[b] < len ? pages_of(len, shift) : 0;
            bool mine = false;
            for (int i = end ? pages_of(kept[b], shift) + tid : 0; i < end; i += kThreads)
                mine |= static_cast<unsigned>(a.p.table[b * a.p.stride + i]) >= static_cast<unsigned>(a.p.num_pages);
            if (end && __syncthreads_or(mine) && tid == 0)
                kept[b] = len;
        }
        __syncthreads();
        x = unused = 0;
        for (int b = b0; b < b1; ++b)
            x = min(x + (kept[b] < a.lens[b] ? pages_of(a.lens[b], shift) - pages_of(kept[b], shift) : 0), most);
        block_before(x, unused, most, most);
        for (int b = b0; b < b1; ++b) {
            x = min(x + (kept[b] < a.lens[b] ? pages_of(a.lens[b], shift) - pages_of(kept[b], shift) : 0), most);
            ahead[b + 1] = static_cast<int>(x);
        }
        __syncthreads();
        given = ahead[a.B];
        fits = given <= a.p.num_pages - count;
        for (int j = tid; fits && j < given; j += kThreads) {
            const int b = owner(ahead, a.B, j);
            a.p.stack[count + given - 1 - j] = a.p.table[b * a.p.stride + pages_of(kept[b], shift) + j - ahead[b]];
        }
    }
    for (int b = tid; b < a.B; b += kThreads)
        a.lens_out[b] = fits ? kept[b] : a.lens[b];
    if (tid == 0 && fits)
        *a.p.count = count + given;
}

static unsigned blocks_for(int64_t items, int num_sms)
{
    const int64_t n = (items + kThreads * kItems - 1) / (kThreads * kItems);
    return static_cast<unsigned>(n < 1 ? 1 : n > num_sms ? num_sms : n);
}

template <class A>
static cudaError_t launch(void (*kern)(A), const A& a, unsigned blocks, int ints, int most_ints, cudaStream_t s)
{
    // More than 48 KB, with what the kernel holds besides, have to be asked for: always
    // the most that a call can need, as another thread's call may be between here and its launch.
    if (ints * 4 > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most_ints * 4);
        if (e != cudaSuccess)
            return e;
    }
    return launch_dependent(kern, dim3(blocks), dim3(kThreads), ints * 4, s, a);
}

// Integers that the kernels' arrays of a call of B sequences take.
static int extend_ints(int B) { return 3 * B + 2; }
static int truncate_ints(int B) { return 2 * B + 1; }

cudaError_t launch_pages_extend(const PagesExtend& a, int num_sms, cudaStream_t s)
{
    return launch(pages_extend_kernel, a, blocks_for(a.T, num_sms), extend_ints(a.B), extend_ints(kPagesMostSeqs), s);
}

cudaError_t launch_pages_truncate(const PagesTruncate& a, int num_sms, cudaStream_t s)
{
    // how many pages go back only the device knows: the most that it could be
    const int64_t most = static_cast<int64_t>(a.B) * a.p.max_pages;
    return launch(pages_truncate_kernel, a, blocks_for(most < a.p.num_pages ? most : a.p.num_pages, num_sms),
                  truncate_ints(a.B), truncate_ints(kPagesMostSeqs), s);
}

}  // namespace w4a8
