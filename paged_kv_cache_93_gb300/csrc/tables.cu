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
// counts is one launch and no round trip.  Every CTA therefore takes the prefix sums
// of the whole batch by itself (into its shared memory) and then fills its share of the
// rows, finding a row's sequence by bisection.  What all CTAs read -- the lengths and
// the stack's height -- is rewritten by the last CTA to finish, which a counter beside
// the height tells; it wraps back to zero by itself.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxBatch = 8192;             // prefix sums of 64 KB

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

// Exclusive prefix sums over the CTA of each thread's pair, and the totals.
__device__ Two cta_scan(Two v, Two &total) {
    __shared__ int64_t sums[2][kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t a = v.a, b = v.b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o);
        const int64_t y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        sums[0][warp] = a;
        sums[1][warp] = b;
    }
    __syncthreads();
    Two before = {0, 0};
    total = {0, 0};
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int64_t x = sums[0][w], y = sums[1][w];
        if (w < warp) {
            before.a += x;
            before.b += y;
        }
        total.a += x;
        total.b += y;
    }
    __syncthreads();               // `sums` is free for the next call
    return {before.a + a - v.a, before.b + b - v.b};
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

__global__ void __launch_bounds__(kThreads) extend_kernel(const TablesArgs a) {
    extern __shared__ int32_t smem[];
    int32_t *cu = smem, *taken = smem + a.batch + 1;      // [batch + 1] each
    pdl_wait();
    pdl_launch_dependents();
    const bool tells = blockIdx.x == 0;                   // raises the batch's flags
    int32_t count = a.state[0];
    if (count < 0 || count > a.num_blocks) {
        if (tells && threadIdx.x == 0) raise_status(a.status, PKV_DEV_BLOCK_ID);
        count = 0;
    }
    const int64_t most = min(int64_t(a.max_blocks) * a.block_size, int64_t(INT32_MAX));
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(int(threadIdx.x) * per, a.batch), b1 = min(b0 + per, a.batch);
    // what sequence b asks for: tokens and blocks (none where its lengths are not valid)
    auto asked = [&](int b, bool flag) -> Two {
        const int32_t len = a.lens[b], n = a.change[b];
        uint32_t bad = 0;
        if (len < 0 || len > most || n < 0) bad = PKV_DEV_SEQ_LEN;
        else if (n > most - len) bad = PKV_DEV_TABLE_RANGE;
        if (bad) {
            if (flag) raise_status(a.status, bad);
            return {0, 0};
        }
        return {n, ceil_div(len + n, a.block_size) - ceil_div(len, a.block_size)};
    };
    Two mine = {0, 0}, total;
    for (int b = b0; b < b1; ++b) {
        const Two x = asked(b, tells);
        mine.a += x.a;
        mine.b += x.b;
    }
    Two at = cta_scan(mine, total);
    if (total.a <= a.rows && total.b <= count) {
        for (int b = b0; b < b1; ++b) {
            cu[b] = int32_t(at.a);
            taken[b] = int32_t(at.b);
            const Two x = asked(b, false);
            at.a += x.a;
            at.b += x.b;
        }
    } else {
        // Not everything fits.  In order: a sequence whose tokens end past the rows
        // brings none; of the others, one whose blocks end past the free ones.  What is
        // refused keeps its place in the sums, so that nothing later overtakes it.
        const Two begin = at;
        int64_t rows_to = begin.a;
        Two again = {0, 0};
        for (int b = b0; b < b1; ++b) {
            const Two x = asked(b, false);
            rows_to += x.a;
            if (x.a > 0 && rows_to > a.rows) {
                if (tells) raise_status(a.status, PKV_DEV_QUERY_RANGE);
            } else {
                again.b += x.b;
            }
        }
        Two blocks_at = cta_scan(again, total);
        Two granted = {0, 0};
        // cu / taken first hold each sequence's own counts
        rows_to = begin.a;
        for (int b = b0; b < b1; ++b) {
            const Two x = asked(b, false);
            rows_to += x.a;
            bool ok = !(x.a > 0 && rows_to > a.rows);
            if (ok) {
                blocks_at.b += x.b;
                if (x.b > 0 && blocks_at.b > count) {
                    ok = false;
                    if (tells) raise_status(a.status, PKV_DEV_NO_BLOCKS);
                }
            }
            cu[b] = ok ? int32_t(x.a) : 0;
            taken[b] = ok ? int32_t(x.b) : 0;
            granted.a += cu[b];
            granted.b += taken[b];
        }
        at = cta_scan(granted, total);
        for (int b = b0; b < b1; ++b) {
            const int32_t n = cu[b], k = taken[b];
            cu[b] = int32_t(at.a);
            taken[b] = int32_t(at.b);
            at.a += n;
            at.b += k;
        }
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
            const int32_t len = a.lens[b], p = len + int32_t(r) - cu[b];
            const int32_t lb = p / a.block_size, held = ceil_div(len, a.block_size);
            const int32_t phys = lb < held ? a.tables[int64_t(b) * a.max_blocks + lb]
                                           : stack[-int64_t(taken[b] + lb - held)];
            position[i] = p;
            if (phys < 0 || phys >= a.num_blocks) raise_status(a.status, PKV_DEV_BLOCK_ID);
            else slot[i] = int64_t(phys) * a.block_size + (p - lb * a.block_size);
        }
        if (r0 + 1 < a.rows) {
            *reinterpret_cast<longlong2 *>(a.positions + r0) = make_longlong2(position[0], position[1]);
            *reinterpret_cast<longlong2 *>(a.slots + r0) = make_longlong2(slot[0], slot[1]);
        } else {
            a.positions[r0] = position[0];
            a.slots[r0] = slot[0];
        }
    }
    // ---- the tables' new entries
    for (int64_t k = thread; k < taken[a.batch]; k += threads) {
        const int b = owner(taken, a.batch, int32_t(k));
        const int32_t held = ceil_div(a.lens[b], a.block_size);
        a.tables[int64_t(b) * a.max_blocks + held + (k - taken[b])] = stack[-k];
    }
    for (int64_t b = thread; b <= a.batch; b += threads) a.cu[b] = cu[b];
    if (!last_cta(a.state)) return;
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
        const int32_t n = cu[b + 1] - cu[b];
        if (n) a.lens[b] += n;
    }
    if (threadIdx.x == 0) a.state[0] = count - taken[a.batch];
}

__global__ void __launch_bounds__(kThreads) trim_kernel(const TablesArgs a) {
    extern __shared__ int32_t smem[];
    int32_t *gone = smem;                                  // [batch + 1]
    pdl_wait();
    pdl_launch_dependents();
    const bool tells = blockIdx.x == 0;
    int32_t count = a.state[0];
    if (count < 0 || count > a.num_blocks) {
        if (tells && threadIdx.x == 0) raise_status(a.status, PKV_DEV_BLOCK_ID);
        count = 0;
    }
    const int64_t most = min(int64_t(a.max_blocks) * a.block_size, int64_t(INT32_MAX));
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(int(threadIdx.x) * per, a.batch), b1 = min(b0 + per, a.batch);
    // whether sequence b gets shorter
    auto cut = [&](int b, bool flag) {
        const int32_t len = a.lens[b], keep = a.change[b];
        if (keep < 0) return false;
        if (len < 0 || len > most || keep > len) {
            if (flag) raise_status(a.status, PKV_DEV_SEQ_LEN);
            return false;
        }
        return keep < len;
    };
    auto blocks = [&](int b) {
        return ceil_div(a.lens[b], a.block_size) - ceil_div(a.change[b], a.block_size);
    };
    Two mine = {0, 0}, total;
    for (int b = b0; b < b1; ++b)
        if (cut(b, tells)) mine.a += blocks(b);
    Two at = cta_scan(mine, total);
    for (int b = b0; b < b1; ++b) {
        gone[b] = int32_t(at.a);
        if (cut(b, false)) at.a += blocks(b);
    }
    if (threadIdx.x == 0) gone[a.batch] = int32_t(total.a);
    __syncthreads();
    const int64_t thread = blockIdx.x * int64_t(kThreads) + threadIdx.x;
    const int64_t threads = int64_t(gridDim.x) * kThreads;
    const int64_t top = count + total.a;
    for (int64_t k = thread; k < total.a; k += threads) {
        const int b = owner(gone, a.batch, int32_t(k));
        const int32_t left = ceil_div(a.change[b], a.block_size);
        const int32_t phys = a.tables[int64_t(b) * a.max_blocks + left + (k - gone[b])];
        if (top - 1 - k < a.num_blocks) a.free_blocks[top - 1 - k] = phys;
    }
    if (!last_cta(a.state)) return;
    for (int b = threadIdx.x; b < a.batch; b += kThreads)
        if (cut(b, false)) a.lens[b] = a.change[b];
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

int launch(void (*kernel)(TablesArgs), const TablesArgs &a, int64_t threads, size_t smem,
           pkv_stream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(2 * (kMaxBatch + 1) * 4));
    if (e != cudaSuccess) return cuda_status(e);
    const int64_t ctas = (threads + kThreads - 1) / kThreads;
    return launch_pdl(kernel, dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>(ctas, sm_count())))),
                      dim3(kThreads), smem, reinterpret_cast<cudaStream_t>(stream), a);
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
    return launch(extend_kernel, a, (int64_t(num_tokens) + 1) / 2, 2 * size_t(batch + 1) * 4, stream);
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
    // a long sequence's blocks are shared among up to 16 CTAs
    const int64_t most = std::min<int64_t>(int64_t(batch) * max_blocks / 16, 16 * kThreads);
    return launch(trim_kernel, a, most, size_t(batch + 1) * 4, stream);
}
