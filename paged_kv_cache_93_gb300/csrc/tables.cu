// tables.cu -- block tables and slot maps kept on the device from request lengths.
//
// The free blocks are a stack: the last of its `count` entries is taken first.  Extend
// gives sequence b, of len_b tokens bringing n_b,
//     need_b = ceil((len_b + n_b) / bs) - ceil(len_b / bs)
// blocks; with `taken_b` the blocks of the sequences before it, the i-th of them is
// free[count - 1 - taken_b - i], so every block is known from prefix sums alone and no
// thread waits for another.  Trim puts blocks back so that it undoes an extend exactly:
// the last sequence's last block first.
//
// Bound: latency.  A step of 1,000 sequences and 40,000 tokens writes 0.8 MB; what
// counts is one launch and few round trips (an extend and the trim that undoes it: 256
// sequences of a token each 7.5 us, 1,000 of up to 512 each 13.5).  Each CTA takes the
// prefix sums of the whole batch by itself, in its shared memory, and then fills its share
// of the rows, finding a row's sequence by bisection.  Up to kRowsAlone rows one CTA does
// it all, and every trim, whose blocks are copied eight a thread at a time: few, as a rule
// (256 sequences of 32K tokens cut to none, 524,288 blocks, take that CTA 309 us).  With
// more rows, what all CTAs read -- the lengths and the stack's height -- is rewritten by
// the last CTA to finish, which a counter beside the height tells; it wraps back to zero by
// itself.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 8192;             // prefix sums and lengths of 96 KB
constexpr int kRowsAlone = 4 * kThreads;

struct TablesArgs {
    int32_t *tables, *lens;
    const int32_t *change;                  // tokens brought, or lengths to keep
    int32_t *free_blocks;
    int32_t *state;                         // [0] free blocks, [1] CTAs that have finished
    int32_t *cu;
    int64_t *positions, *slots;
    uint32_t *status;
    int32_t batch, max_blocks, block_size, num_blocks, rows;
};

struct Two {
    int64_t a, b;
};

// Inclusive prefix sums over the warp.
__device__ __forceinline__ Two warp_scan(Two v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v.a, o);
        const int64_t y = __shfl_up_sync(0xffffffffu, v.b, o);
        if (lane >= o) {
            v.a += x;
            v.b += y;
        }
    }
    return v;
}

// Exclusive prefix sums over the CTA of each thread's pair, and the totals.
__device__ Two cta_scan(Two v, Two &total) {
    static_assert(kThreads == 32 * 32, "a warp scans the warps' sums");
    __shared__ Two sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Two upto = warp_scan(v);
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    if (warp == 0) sums[lane] = warp_scan(sums[lane]);
    __syncthreads();
    const Two before = warp ? sums[warp - 1] : Two{0, 0};
    total = sums[31];
    __syncthreads();               // `sums` is free for the next call
    return {before.a + upto.a - v.a, before.b + upto.b - v.b};
}

// The last entry of the rising list first[0 .. n] that is <= x (first[0] <= x < first[n]).
__device__ __forceinline__ int owner(const int32_t *first, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// True in the one CTA that every other one has finished before.
__device__ bool last_cta(int32_t *state) {
    __shared__ uint32_t s_last;
    if (gridDim.x == 1) {
        __syncthreads();
        return true;
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = atomicInc(reinterpret_cast<unsigned int *>(state) + 1, gridDim.x - 1) ==
                 gridDim.x - 1;
    __syncthreads();
    __threadfence();
    return s_last != 0;
}

__device__ __forceinline__ int32_t ceil_div(int32_t x, int32_t n) {
    return int32_t((uint32_t(x) + uint32_t(n) - 1) / uint32_t(n));
}

// The lengths and changes into L2 while the kernel before this one ends.
__device__ __forceinline__ void prefetch_lengths(const TablesArgs &a) {
    const int64_t at = threadIdx.x * 128, bytes = int64_t(a.batch) * 4;
    if (blockIdx.x == 0 && at < bytes) {
        asm volatile("prefetch.global.L2 [%0];"
                     ::"l"(reinterpret_cast<const char *>(a.lens) + at));
        asm volatile("prefetch.global.L2 [%0];"
                     ::"l"(reinterpret_cast<const char *>(a.change) + at));
    }
}

__device__ __forceinline__ int32_t stack_height(const TablesArgs &a) {
    const int32_t count = a.state[0];
    if (count >= 0 && count <= a.num_blocks) return count;
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(a.status, PKV_DEV_BLOCK_ID);
    return 0;
}

__global__ void __launch_bounds__(kThreads) extend_kernel(const TablesArgs a) {
    extern __shared__ int32_t smem[];
    // [batch + 1] each; first what each sequence brings, then the sums
    int32_t *cu = smem, *taken = smem + a.batch + 1, *lens = taken + a.batch + 1;
    prefetch_lengths(a);
    pdl_wait();
    pdl_launch_dependents();
    const bool tells = blockIdx.x == 0;                   // raises the batch's flags
    const int32_t count = stack_height(a);
    const int64_t most = min(int64_t(a.max_blocks) * a.block_size, int64_t(INT32_MAX));
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(int(threadIdx.x) * per, a.batch), b1 = min(b0 + per, a.batch);
    // tokens and blocks that each sequence asks for (none where its lengths are not valid)
    Two mine = {0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const int32_t len = a.lens[b], n = a.change[b];
        uint32_t bad = 0;
        if (len < 0 || len > most || n < 0) bad = PKV_DEV_SEQ_LEN;
        else if (n > most - len) bad = PKV_DEV_TABLE_RANGE;
        if (bad && tells) raise_status(a.status, bad);
        lens[b] = len;
        cu[b] = bad ? 0 : n;
        taken[b] = bad ? 0 : ceil_div(len + n, a.block_size) - ceil_div(len, a.block_size);
        mine.a += cu[b];
        mine.b += taken[b];
    }
    Two at = cta_scan(mine, total);
    if (total.a > a.rows || total.b > count) {
        // Not everything fits.  In order: a sequence whose tokens end past the rows
        // brings none; of the others, one whose blocks end past the free ones.  What is
        // refused keeps its place in the sums, so that nothing later overtakes it.
        Two again = {0, 0};
        for (int b = b0; b < b1; ++b) {
            const int32_t n = cu[b];
            at.a += n;
            if (n > 0 && at.a > a.rows) {
                if (tells) raise_status(a.status, PKV_DEV_QUERY_RANGE);
                cu[b] = taken[b] = 0;
            }
            again.b += taken[b];
        }
        at = cta_scan(again, total);
        Two granted = {0, 0};
        for (int b = b0; b < b1; ++b) {
            const int32_t k = taken[b];
            at.b += k;
            if (k > 0 && at.b > count) {
                if (tells) raise_status(a.status, PKV_DEV_NO_BLOCKS);
                cu[b] = taken[b] = 0;
            }
            granted.a += cu[b];
            granted.b += taken[b];
        }
        at = cta_scan(granted, total);
    }
    for (int b = b0; b < b1; ++b) {
        const int32_t n = cu[b], k = taken[b];
        cu[b] = int32_t(at.a);
        taken[b] = int32_t(at.b);
        at.a += n;
        at.b += k;
    }
    if (threadIdx.x == 0) {
        cu[a.batch] = int32_t(total.a);
        taken[a.batch] = int32_t(total.b);
    }
    __syncthreads();
    const int64_t thread = blockIdx.x * int64_t(kThreads) + threadIdx.x;
    const int64_t threads = int64_t(gridDim.x) * kThreads;
    const int32_t *stack = a.free_blocks + count - 1;      // the k-th block taken: stack[-k]
    // ---- the rows, two at a time
    const int32_t live = cu[a.batch];
    for (int64_t r0 = 2 * thread; r0 < a.rows; r0 += 2 * threads) {
        int64_t position[2] = {-1, -1}, slot[2] = {-1, -1};
        int b = r0 < live ? owner(cu, a.batch, int32_t(r0)) : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t r = r0 + i;
            if (r >= live) break;
            while (r >= cu[b + 1]) ++b;
            const int32_t len = lens[b], p = len + int32_t(r) - cu[b];
            const int32_t lb = p / a.block_size, held = ceil_div(len, a.block_size);
            const int32_t phys = lb < held ? a.tables[int64_t(b) * a.max_blocks + lb]
                                           : stack[-int64_t(taken[b] + lb - held)];
            position[i] = p;
            if (phys < 0 || phys >= a.num_blocks) raise_status(a.status, PKV_DEV_BLOCK_ID);
            else slot[i] = int64_t(phys) * a.block_size + (p - lb * a.block_size);
        }
        if (r0 + 1 < a.rows) {
            *reinterpret_cast<longlong2 *>(a.positions + r0) =
                make_longlong2(position[0], position[1]);
            *reinterpret_cast<longlong2 *>(a.slots + r0) = make_longlong2(slot[0], slot[1]);
        } else {
            a.positions[r0] = position[0];
            a.slots[r0] = slot[0];
        }
    }
    // ---- the tables' new entries
    for (int64_t k = thread; k < taken[a.batch]; k += threads) {
        const int b = owner(taken, a.batch, int32_t(k));
        const int32_t held = ceil_div(lens[b], a.block_size);
        a.tables[int64_t(b) * a.max_blocks + held + (k - taken[b])] = stack[-k];
    }
    for (int64_t b = thread; b <= a.batch; b += threads) a.cu[b] = cu[b];
    if (!last_cta(a.state)) return;
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
        const int32_t n = cu[b + 1] - cu[b];
        if (n) a.lens[b] = lens[b] + n;
    }
    if (threadIdx.x == 0) a.state[0] = count - taken[a.batch];
}

// One CTA.
__global__ void __launch_bounds__(kThreads) trim_kernel(const TablesArgs a) {
    extern __shared__ int32_t smem[];
    // [batch + 1] each: blocks given back, then their sums; the blocks that are kept
    int32_t *gone = smem, *left = smem + a.batch + 1;
    prefetch_lengths(a);
    pdl_wait();
    pdl_launch_dependents();
    const int32_t count = stack_height(a);
    const int64_t most = min(int64_t(a.max_blocks) * a.block_size, int64_t(INT32_MAX));
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(int(threadIdx.x) * per, a.batch), b1 = min(b0 + per, a.batch);
    Two mine = {0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const int32_t len = a.lens[b], keep = a.change[b];
        gone[b] = 0;
        if (keep < 0) continue;
        if (len < 0 || len > most || keep > len) {
            raise_status(a.status, PKV_DEV_SEQ_LEN);
            continue;
        }
        left[b] = ceil_div(keep, a.block_size);
        gone[b] = ceil_div(len, a.block_size) - left[b];
        mine.a += gone[b];
        if (keep < len) a.lens[b] = keep;
    }
    Two at = cta_scan(mine, total);
    for (int b = b0; b < b1; ++b) {
        const int32_t k = gone[b];
        gone[b] = int32_t(at.a);
        at.a += k;
    }
    if (threadIdx.x == 0) gone[a.batch] = int32_t(total.a);
    __syncthreads();
    const int64_t top = count + total.a;
    constexpr int kAhead = 8;
    for (int64_t k0 = threadIdx.x; k0 < total.a; k0 += kThreads * kAhead) {
        int32_t phys[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t k = k0 + u * kThreads;
            if (k < total.a) {
                const int b = owner(gone, a.batch, int32_t(k));
                phys[u] = a.tables[int64_t(b) * a.max_blocks + left[b] + (k - gone[b])];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t to = top - 1 - (k0 + u * kThreads);
            if (k0 + u * kThreads < total.a && to < a.num_blocks) a.free_blocks[to] = phys[u];
        }
    }
    if (threadIdx.x == 0) {
        if (top > a.num_blocks) raise_status(a.status, PKV_DEV_BLOCK_ID);
        a.state[0] = int32_t(min(top, int64_t(a.num_blocks)));
    }
}

int check(int32_t block_size, int32_t num_blocks, int32_t batch, int32_t max_blocks) {
    if (block_size < 1 || block_size > 256 || num_blocks <= 0 || batch < 0 || max_blocks < 0)
        return PKV_ERR_INVALID_ARG;
    if (batch > kMaxBatch || int64_t(batch) * max_blocks > INT32_MAX) return PKV_ERR_SHAPE;
    return PKV_OK;
}

int launch(void (*kernel)(TablesArgs), const TablesArgs &a, int64_t ctas, pkv_stream_t stream) {
    // once a device and thread: room for the longest prefix sums
    static thread_local int configured = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured != dev) {
        for (auto k : {extend_kernel, trim_kernel})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(3 * (kMaxBatch + 1) * 4));
        if (e == cudaSuccess) configured = dev;
    }
    if (e != cudaSuccess) return cuda_status(e);
    return launch_pdl(kernel, dim3(unsigned(std::min<int64_t>(ctas, sm_count()))), dim3(kThreads),
                      3 * size_t(a.batch + 1) * 4, reinterpret_cast<cudaStream_t>(stream), a);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_extend_sequences(int32_t block_size, int32_t num_blocks, int32_t *block_tables,
                                    int32_t *seq_lens, const int32_t *new_lens, int32_t batch,
                                    int32_t max_blocks, int32_t *free_blocks, int32_t *pool_state,
                                    int32_t num_tokens, int32_t *cu_q_lens, int64_t *positions,
                                    int64_t *slot_mapping, pkv_stream_t stream) {
    const int st = check(block_size, num_blocks, batch, max_blocks);
    if (st == PKV_ERR_INVALID_ARG || num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (st != PKV_OK) return st;
    if (batch == 0 && num_tokens == 0 && !cu_q_lens) return PKV_OK;
    if ((batch > 0 && (!block_tables || !seq_lens || !new_lens)) || !free_blocks || !pool_state ||
        !cu_q_lens || (num_tokens > 0 && (!positions || !slot_mapping)))
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(positions) || !aligned16(slot_mapping)) return PKV_ERR_ALIGNMENT;
    TablesArgs a = {};
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    a.tables = block_tables;
    a.lens = seq_lens;
    a.change = new_lens;
    a.free_blocks = free_blocks;
    a.state = pool_state;
    a.cu = cu_q_lens;
    a.positions = positions;
    a.slots = slot_mapping;
    a.batch = batch;
    a.max_blocks = max_blocks;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.rows = num_tokens;
    // (two rows a thread)
    const int64_t ctas =
        num_tokens <= kRowsAlone ? 1 : (int64_t(num_tokens) + 2 * kThreads - 1) / (2 * kThreads);
    return launch(extend_kernel, a, ctas, stream);
}

extern "C" int pkv_trim_sequences(int32_t block_size, int32_t num_blocks,
                                  const int32_t *block_tables, int32_t *seq_lens,
                                  const int32_t *keep_lens, int32_t batch, int32_t max_blocks,
                                  int32_t *free_blocks, int32_t *pool_state, pkv_stream_t stream) {
    const int st = check(block_size, num_blocks, batch, max_blocks);
    if (st != PKV_OK) return st;
    if (batch == 0) return PKV_OK;
    if (!block_tables || !seq_lens || !keep_lens || !free_blocks || !pool_state)
        return PKV_ERR_INVALID_ARG;
    TablesArgs a = {};
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    a.tables = const_cast<int32_t *>(block_tables);
    a.lens = seq_lens;
    a.change = keep_lens;
    a.free_blocks = free_blocks;
    a.state = pool_state;
    a.batch = batch;
    a.max_blocks = max_blocks;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    return launch(trim_kernel, a, 1, stream);
}
