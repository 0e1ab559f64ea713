// chunk_tc.cu -- attention of ragged chunks of new tokens over the paged cache
// on the 5th-generation tensor cores of sm_103a: bf16 caches with head dims 64
// or 128, E4M3 caches with head dim 128.
//
// The rows of one KV head -- (token, query head of the group) pairs, token
// major -- are packed into tiles of 128 (tokens_per_tile = 128 / group, so an odd
// group wastes the remainder).  With m a reference of the row,
//   S[128 rows x 128 keys] = Q_tile . K_tile^T             (tcgen05, fp32 in TMEM)
//   P = 2^((S - m) scale log2 e), l += row sums of P       (CUDA cores, one thread a row)
//   O[128 rows x D]       += P . V_tile                    (tcgen05, P read from TMEM)
// and out = O / l, lse = m scale + ln l.  P is rounded to bf16 for the second
// product (its sum is taken before the rounding, in fp32): one bf16 term is
// what the bf16 output resolves.  E4M3 caches: Q goes as two E4M3 terms, the
// second the rounding residual of the first (a bf16 element fits them exactly
// unless it is far below its row's largest), so the stored keys feed the tensor
// cores as they are, in the time of one bf16 product; the values are widened to
// fp16, which holds them exactly, and P is rounded to fp16.  (Two E4M3 terms of P cost
// the softmax threads six conversions for four scores: 1,000 tokens over 17K keys went
// from 650 to 502 us when only that changed.)
//
// Work item = (block of up to 2 tiles' tokens of a sequence, KV head, all of its
// key tiles or a run of them), given out by plan_kernel:
//  - a pair item has two row tiles A and B that read the same keys: while the
//    tensor cores work for one, the CUDA cores take the softmax of the other;
//  - a block of at most one tile's tokens is a split item: A and B are the
//    same rows over the first and second half of the item's key tiles.
// A cut item's partial (O / l, lse), and the two halves' of a split item, go to
// the workspace and chunk_merge_kernel joins them.
//
// Roles, one CTA an SM: warps 0-3 softmax and epilogue of A, warps 4-7 of B, one
// thread a row, warp 8 MMA issue, warp 9 TMA; head dim 64: warps 10 and 11, E4M3:
// warps 12-15, see to the value tiles.  TMEM, all 512 columns: S_A S_B O_A O_B, P
// over S.  The MMAs of one thread run in order, so S may be overwritten by a
// score product once the value product that reads P there is issued.  Every wait
// is bounded.
//
// What bounds it (2,048 tokens over 32K keys, 32 heads over 8, 679 us, 1.57 PFLOP/s,
// 0.81 of the measured bf16 rate): a step of a pair item -- four products of 512
// cycles -- takes 2,860 cycles.  The products of a half wait for its softmax, that
// for the scores before, and what the issuing thread does between two products
// (waits, commits) leaves the tensor cores idle.  A third S buffer, which head dim
// 64 has room for, so that a half's next scores are there early, changed nothing
// (241 us either way, an 8K prompt under a window of 1,024).  Single tokens read
// 4.8 TB/s: the ring holds little more than a step of a split item.
//
// Keys are walked in absolute 128-key tiles.  Under a window the tiles
// between the sinks and the first row's window are skipped; in a tile only
// the blocks that some row of the item sees are copied, and the value rows of
// keys no row sees are zeroed in shared memory, so stale bits (0 * NaN) never
// reach O.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_math.cuh"
#include "pkv_pipeline.cuh"
#include "pkv_tcgen05_ts.cuh"

namespace pkv {
namespace {

constexpr int kRows = 128;               // query rows per tile (TMEM lanes)
constexpr int kKeys = 128;               // keys per tile
constexpr int kMmaWarp = 8, kLoadWarp = 9, kWidenWarp = 12;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;          // O_A, O_B; S_A, S_B at 0 and 128
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// E4M3 caches: probabilities are taken 2^kLift times as large as against the reference.
// fp16 steps by 2^-24 at the least, so one loses bits from 2^-14 and vanishes at 2^-25;
// with a lift of 8 that is 2^-22 (15.2 nats) and 2^-33 (22.9) of the row's largest, and
// 64 that equal it add up to 2^14, below kMost.
constexpr float kLift = 8.f;

template <int D, bool E4>
struct Cfg {
    static_assert(D == 64 || D == 128, "head dims of one or two 128-byte column blocks");
    static_assert(!E4 || D == 128, "E4M3 rows fill a 128-byte swizzle row");
    static constexpr int kElem = E4 ? 1 : 2;
    // Three warp groups, four with the one that widens values.  Registers a thread:
    // launched with 168 (128), the softmax groups then take kSoftRegs, the others
    // keep kOtherRegs; the sums are those of the launch or less.
    static constexpr int kThreads = E4 ? 512 : 384;
    static constexpr int kSoftRegs = E4 ? 184 : 200, kOtherRegs = E4 ? 72 : 104;
    static constexpr int kWideners = 4;                             // warps
    static constexpr uint32_t kHalfTile = kRows * 128;              // [128 rows][128 B]
    static constexpr uint32_t kQTile = E4 ? 2 * kHalfTile : kRows * D * 2;
    static constexpr uint32_t kStage = kKeys * D * kElem;           // a K or V tile
    static constexpr int kStages = E4 ? 6 : kStage == 32768 ? 5 : 10;
    // Who makes the value rows 0 that no row of an item sees.  Head dim 64, whose
    // softmax bounds a step: the two idle warps (an 8K prompt under a window of 1,024
    // 250 -> 241 us); head dim 128, where a tile's way to the tensor cores counts: the
    // softmax warps (8K prompt 388 -> 380 us); E4M3: the warps that widen.
    static constexpr bool kTended = D == 64;
    // How a warp that gave up keeps from arriving: by a vote a tile, or by a test before
    // each arrival (8K prompt under a window, head dim 64: 240.5 us against 243.2, and
    // 241 without either; 8K prompt, head dim 128: 386 against 380, and 380; FP8 chunk:
    // 439 against 434, and 431).
    static constexpr bool kEndsItem = D == 64;
    static constexpr uint32_t kWide = kKeys * D * 2;                // a V tile in 16 bits
    static constexpr uint32_t kOffQ = 1024;
    static constexpr uint32_t kOffRing = kOffQ + 2 * kQTile;
    static constexpr uint32_t kOffWide = kOffRing + kStages * kStage;
    static constexpr uint32_t kSmem = 1024 + kOffWide + (E4 ? 2 * kWide : 0);
    // The sum of 64 probabilities past which a row's reference rises.  bf16: far
    // below overflow of the sums over 2^30 keys and of products with values up to
    // 2^80.  fp16: none of them passes 65,504, its largest number.
    static constexpr float kMost = E4 ? 65504.f : 1048576.f;
    static constexpr uint32_t kIdS = E4 ? tc::idesc_e4m3_f32(kRows, kKeys, 0, 0)
                                        : tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
    static constexpr uint32_t kIdO = E4 ? tc::idesc_f16_f32(kRows, D, 0, 1)
                                        : tc::idesc_bf16_f32(kRows, D, 0, 1);
};

// mbarrier slots
constexpr int kBarFull = 0;              // + stage (at most 10)
constexpr int kBarEmpty = 10;            // + stage.  E4M3: two arrivals, of a value tile the
                                         // widening warps', of a key tile the producer's
                                         // own and the commit
constexpr int kBarQFull = 20;
constexpr int kBarQEmpty = 21;           // commit: the item's score products are done
constexpr int kBarSFull = 22;            // + half: scores written (commit)
constexpr int kBarPFull = 24;            // + 2 part + half: probabilities of 64 keys written
                                         // (128 arrivals)
constexpr int kBarPvDone = 28;           // + half: the item's value products done (commit)
constexpr int kBarP0Done = 30;           // + half: value product of a tile's first 64 keys done
constexpr int kBarOEmpty = 32;           // + half: O read out (128 arrivals)
constexpr int kBarDrain = 34;
constexpr int kBarWideFull = 35;         // + buffer: values widened (128 arrivals)
constexpr int kBarWideEmpty = 37;        // + buffer: their value products done (commit)
constexpr int kBarReady = 39;            // + stage: a tile is in place, the unseen rows of a V
                                         // tile 0 (kTended; 2 arrivals)
constexpr uint32_t kOffSlot = 49 * 8;
constexpr uint32_t kOffFlag = kOffSlot + 4;

// A query block: up to 2 tiles' tokens of a sequence (all KV heads alike).
struct __align__(16) Block {
    int32_t b, qrow, pos, ntok;          // sequence; row of q and position of its first token
    int32_t tiles, steps, prow, work;    // key tiles; steps of the whole; partial rows of KV
                                         // head 0 when taken whole as a split item, or -1;
                                         // steps in pair items' steps (split_work)
};
// What a CTA does at a time: some steps of a (block, KV head).
struct __align__(16) Item {
    int32_t b, qrow, pos, ntok;
    int32_t v0, na, nb, prow;            // first key tile, tiles of A and B; partial row or -1
    int32_t g, split, pad0, pad1;
};
// A (block, KV head) cut over several CTAs: its first piece's partials are in slot
// ctas + cta, the others' in the slots of the `more` CTAs that follow.
struct __align__(16) Cut {
    int32_t block, g, cta, more;
};
struct Plan {                            // device pointers into the workspace
    int32_t *header;
    Block *blocks;                       // in the order of the work
    int32_t *before;                     // cost of the blocks before each
    int32_t *first;                      // [batch + 1] query blocks before a sequence
    int32_t *split;                      // blocks taken as split items with partials
    uint8_t *is_cut;                     // [(block, KV head)] of the second part of the work
    Cut *cuts;                           // [ctas]
    int32_t *piece0;                     // [ctas + 1] first piece of a CTA
    Item *pieces;
    float *o_part, *lse_part;            // [partial rows][D], [partial rows]
    int32_t ctas, slot_rows;             // rows of a slot; slots come first, 2 for each CTA
};
constexpr int kHdrBlocks = 0;            // query blocks
constexpr int kHdrRounds = 1;            // whole items of every CTA
constexpr int kHdrByHead = 2;            // work order: KV head major
constexpr int kHdrSplit = 3;             // entries of `split`
constexpr int kHdrCuts = 4;              // entries of `cuts`
constexpr int kHdrSplitRows = 5;         // most rows of an entry of `split`

struct Shape {
    int32_t group, tokens_per_tile;
};

// The key tiles a query block sees: virtual tiles 0 .. count - 1, of which
// the first `sink_tiles` are tiles 0.., the others shifted by `gap`.
struct Tiles {
    int32_t count, sink_tiles, gap, lo;  // lo: first key in the window of the first token
};
__device__ __forceinline__ Tiles tiles_of(int32_t pos, int32_t ntok, int32_t window,
                                          int32_t sinks) {
    Tiles t;
    const int32_t last = pos + ntok - 1;
    const int32_t end = last < 0 ? 0 : last / kKeys + 1;
    t.lo = window > 0 ? max(0, pos - window + 1) : 0;
    const int32_t w0 = t.lo / kKeys;
    t.sink_tiles = min((sinks + kKeys - 1) / kKeys, w0);
    t.gap = w0 - t.sink_tiles;
    t.count = max(0, end - t.gap);
    return t;
}

// Steps s0 .. s1 - 1 of a block: a pair item takes one key tile a step, a split
// item two, its half A the first of its tiles.
__device__ __forceinline__ Item item_of(const Block &q, int32_t g, int32_t s0, int32_t s1,
                                        int32_t tpt, int32_t prow) {
    Item r;
    r.b = q.b;
    r.qrow = q.qrow;
    r.pos = q.pos;
    r.ntok = q.ntok;
    r.g = g;
    r.prow = prow;
    r.split = q.ntok <= tpt;
    if (r.split) {
        r.v0 = 2 * s0;
        const int32_t tiles = min(q.tiles, 2 * s1) - 2 * s0;
        r.na = (tiles + 1) >> 1;
        r.nb = tiles >> 1;
    } else {
        r.v0 = s0;
        r.na = r.nb = s1 - s0;
    }
    r.pad0 = r.pad1 = 0;
    return r;
}

// Work order: (block r, KV head g) <-> index.
__device__ __forceinline__ void item_at(int32_t idx, bool by_head, int32_t nblocks, int32_t hkv,
                                        int32_t &r, int32_t &g) {
    const uint32_t n = by_head ? nblocks : hkv, q = uint32_t(idx) / n;
    g = by_head ? q : idx - q * n;
    r = by_head ? idx - q * n : q;
}
// The whole item CTA `cta` takes in round k: forth and back, so that the CTAs'
// sums of a falling sequence stay near.
__device__ __forceinline__ int32_t round_item(int32_t k, int32_t cta, int32_t ctas) {
    return k * ctas + (k & 1 ? ctas - 1 - cta : cta);
}

// ------------------------------------------------------------------- the plan
constexpr int kPlanThreads = 256;        // all of them run every step: more only slow it
                                         // down (1,024: twice the time)
constexpr int kMaxCtas = kPlanThreads;
// Costs in steps of an item beside its own, measured (2,048 tokens over 32K
// keys): an item's start and end, and those of a piece of a cut item, whose
// partial results (128 KB) go through memory; pieces of fewer steps than
// kSnap are left to the neighbour.
constexpr int kItemCost = 3, kPieceCost = 6, kSnap = 6;
// A step of a split item moves and handles two key tiles, a pair item's one: 1.5
// times the cost (E4M3, keys in L2: 5,200 cycles against 3,250).  And back.
__device__ __forceinline__ int32_t split_work(int32_t steps) { return steps + (steps >> 1); }
__device__ __forceinline__ int32_t split_steps(int32_t work) { return work - work / 3; }

// Inclusive scans of three numbers over the CTA's threads; the sums go to
// `total`.
__device__ __forceinline__ int3 block_scan(int3 v, int3 *warp_sums, int3 &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto warp_scan = [&](int3 &u) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, u.x, o);
            const int y = __shfl_up_sync(0xffffffffu, u.y, o);
            const int z = __shfl_up_sync(0xffffffffu, u.z, o);
            if (lane >= o) {
                u.x += x;
                u.y += y;
                u.z += z;
            }
        }
    };
    warp_scan(v);
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int3 s = lane < kPlanThreads / 32 ? warp_sums[lane] : make_int3(0, 0, 0);
    warp_scan(s);                        // by every warp: no barrier after it
    total = make_int3(__shfl_sync(0xffffffffu, s.x, 31), __shfl_sync(0xffffffffu, s.y, 31),
                      __shfl_sync(0xffffffffu, s.z, 31));
    const int from = (warp + 31) & 31;
    const int x = __shfl_sync(0xffffffffu, s.x, from), y = __shfl_sync(0xffffffffu, s.y, from);
    const int z = __shfl_sync(0xffffffffu, s.z, from);
    return warp ? make_int3(v.x + x, v.y + y, v.z + z) : v;
}

// One CTA makes the plan.  The work -- every (query block, KV head), longest
// first unless they are nearly alike -- is given out in two parts: rounds of
// whole items, one to each CTA, as long as no CTA passes its even share T; then
// the rest, laid end to end, cut at the points where the CTAs' remaining
// capacities T - load end.  So few blocks over long contexts are cut over all
// CTAs evenly, and many blocks are mostly whole.  Nearly alike blocks are
// ordered by KV head, which keeps the keys that are read at one time few.
//
// Up to kInShared sequences and query blocks its tables are kept in shared
// memory (a dependent load from L2 costs more than a scan); more blocks than
// that are not sorted: the capacities even out what is left.
constexpr int kInShared = 1024;          // (s_key: ten bits)

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const ChunkArgs a, const Plan plan, const Shape sh) {
    __shared__ int3 warp_sums[32];
    __shared__ int32_t s_first[kInShared + 1], s_cu[kInShared + 1], s_len[kInShared];
    __shared__ int32_t s_before[kInShared + 1], s_work[kInShared], s_prow[kInShared];
    __shared__ __align__(16) uint32_t s_key[kInShared];          // low 10 bits: the block at a place
    __shared__ int32_t cut_idx[kMaxCtas + 1], cut_step[kMaxCtas + 1];
    __shared__ int32_t s_max, s_min, s_split_rows, s_rounds;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const int32_t hkv = a.cache.num_kv_heads, tpt = sh.tokens_per_tile, per = 2 * tpt;
    const int32_t ctas = plan.ctas;
    int3 total;

    // ---- query blocks before each sequence
    const bool few_seqs = a.batch <= kInShared;
    bool bad = false;
    int32_t nblocks = 0;
    if (tid == 0) {
        s_max = 0;
        s_min = INT_MAX;
        s_split_rows = 0;
        s_rounds = INT_MAX;
    }
    for (int base = 0; base < a.batch; base += kPlanThreads) {
        const int b = base + tid;
        int32_t nq = 0, x = 0, y = 0, L = 0;
        if (b < a.batch) {
            x = a.cu_q_lens[b];
            y = a.cu_q_lens[b + 1];
            L = a.seq_lens[b];
            if (x < 0 || y < x || y > a.num_tokens) bad = true;
            else nq = uint32_t(y - x + per - 1) / uint32_t(per);
            if (L < 0 || L > int64_t(a.max_blocks) * a.cache.block_size) {
                raise_status(a.status, PKV_DEV_SEQ_LEN);
                L = 0;
            } else if (!bad && L < y - x) {
                raise_status(a.status, PKV_DEV_SEQ_LEN);
            }
        }
        if (__syncthreads_or(bad)) {
            if (tid == 0) {
                raise_status(a.status, PKV_DEV_QUERY_RANGE);
                plan.header[kHdrBlocks] = plan.header[kHdrRounds] = plan.header[kHdrSplit] =
                    plan.header[kHdrCuts] = 0;
            }
            for (int j = tid; j <= ctas; j += kPlanThreads) plan.piece0[j] = 0;
            return;
        }
        const int3 incl = block_scan(make_int3(nq, 0, 0), warp_sums, total);
        if (b < a.batch) {
            const int32_t before = nblocks + incl.x - nq;
            if (few_seqs) {
                s_first[b] = before;
                s_cu[b] = x;
                s_cu[b + 1] = y;
                s_len[b] = L;
            } else {
                plan.first[b] = before;
            }
        }
        nblocks += total.x;
    }
    if (tid == 0) (few_seqs ? s_first : plan.first)[a.batch] = nblocks;
    __syncthreads();
    const bool few_blocks = nblocks <= kInShared;

    auto block_of = [&](int i) {
        const int32_t *first = few_seqs ? s_first : plan.first;
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid;
            else hi = mid;
        }
        Block q;
        q.b = lo;
        const int32_t *cu = few_seqs ? s_cu : a.cu_q_lens;
        const int32_t q0 = cu[lo], n = cu[lo + 1] - q0, t0 = (i - first[lo]) * per;
        int32_t L = few_seqs ? s_len[lo] : a.seq_lens[lo];
        if (!few_seqs && (L < 0 || L > int64_t(a.max_blocks) * a.cache.block_size)) L = 0;
        q.qrow = q0 + t0;
        q.pos = L - n + t0;
        q.ntok = min(per, n - t0);
        q.tiles = tiles_of(q.pos, q.ntok, a.window, a.sinks).count;
        q.steps = q.ntok <= tpt ? (q.tiles + 1) >> 1 : q.tiles;
        q.prow = -1;
        q.work = q.ntok <= tpt ? split_work(q.steps) : q.steps;
        return q;
    };

    // ---- the blocks in order
    int32_t most = 0, least = INT_MAX;
    for (int i = tid; i < nblocks; i += kPlanThreads) {
        const Block q = block_of(i);
        if (few_blocks) s_key[i] = uint32_t((1 << 20) - 1 - min(q.work, (1 << 20) - 1)) << 10 | i;
        most = max(most, q.work);
        least = min(least, q.work);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    if ((tid & 31) == 0) {
        atomicMax(&s_max, most);
        atomicMin(&s_min, least);
    }
    __syncthreads();
    const bool by_head = s_max - s_min <= s_max / 4;       // nearly alike
    const int32_t n_items = nblocks * hkv;       // below 2^29 as the query rows are
    // costs in units of 2^shift steps, so that their sum stays below 2^30
    int32_t shift = 0;
    while (float(s_max + kItemCost) * float(n_items) > float(1 << 30) * float(1u << shift)) ++shift;
    auto cost_of = [&](int32_t work) { return ((work + kItemCost) >> shift) + (shift > 0); };
    const int32_t item_cost = cost_of(0), piece_cost = (kPieceCost >> shift) + (shift > 0);
    if (few_blocks && !by_head && n_items > ctas) {
        // a key's place is the number of smaller ones (keys differ: the block is in them)
        for (int i = nblocks + tid; i < (nblocks + 3 & ~3); i += kPlanThreads)
            s_key[i] = 0xffffffffu;
        __syncthreads();
        uint32_t key[kInShared / kPlanThreads];
        int place[kInShared / kPlanThreads];
#pragma unroll
        for (int u = 0; u < kInShared / kPlanThreads; ++u) {
            const int i = tid + u * kPlanThreads;
            place[u] = -1;
            if (i >= nblocks) continue;
            key[u] = s_key[i];
            int n = 0;
            for (int j = 0; j < nblocks; j += 4) {
                const uint4 k = *reinterpret_cast<const uint4 *>(s_key + j);
                n += (k.x < key[u]) + (k.y < key[u]) + (k.z < key[u]) + (k.w < key[u]);
            }
            place[u] = n;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kInShared / kPlanThreads; ++u)
            if (place[u] >= 0) s_key[place[u]] = key[u];
        __syncthreads();
    }
    auto ordered = [&](int r) { return block_of(few_blocks ? int(s_key[r] & 1023u) : r); };
    int32_t cost_all = 0, nsplit = 0, part_rows = 2 * ctas * plan.slot_rows;
    for (int base = 0; base < nblocks; base += kPlanThreads) {
        const int i = base + tid;
        Block q = {};
        const bool in = i < nblocks;
        if (in) q = ordered(i);
        const bool halves = in && q.ntok <= tpt && q.tiles > 1;
        const int32_t cost = in ? cost_of(q.work) : 0;
        const int32_t rows = halves ? 2 * q.ntok * sh.group * hkv : 0;
        const int3 v = block_scan(make_int3(cost, halves, rows), warp_sums, total);
        if (in) {
            const int32_t before = cost_all + v.x - cost;
            if (halves) {
                atomicMax(&s_split_rows, q.ntok * sh.group);
                plan.split[nsplit + v.y - 1] = i;
                q.prow = part_rows + v.z - rows;
            }
            plan.blocks[i] = q;
            if (few_blocks) {
                s_before[i] = before;
                s_work[i] = q.work * 2 + (q.ntok <= tpt);
                s_prow[i] = q.prow;
            } else {
                plan.before[i] = before;
            }
        }
        cost_all += total.x;
        nsplit += total.y;
        part_rows += total.z;
    }
    if (tid == 0) (few_blocks ? s_before : plan.before)[nblocks] = cost_all;
    __syncthreads();
    const int32_t *before = few_blocks ? s_before : plan.before;
    auto work_at = [&](int r) { return few_blocks ? s_work[r] >> 1 : plan.blocks[r].work; };

    // ---- whole rounds
    const int32_t share = uint32_t(cost_all * hkv) / uint32_t(ctas) + 1 + piece_cost;
    // (each thread on its own: the most rounds its CTA takes; the least of them counts)
    const int32_t most_rounds = n_items / ctas;
    auto round_cost = [&](int k) {
        int32_t r, g;
        item_at(round_item(k, tid, ctas), by_head, nblocks, hkv, r, g);
        return cost_of(work_at(r));
    };
    if (tid < ctas) {
        int32_t sum = 0, k = 0;
        for (; k < most_rounds; ++k) {
            sum += round_cost(k);
            if (sum > share) break;
        }
        if (k < most_rounds) atomicMin(&s_rounds, k);
    }
    __syncthreads();
    const int32_t rounds = min(s_rounds, most_rounds);
    int32_t load = 0;
    if (tid < ctas)
        for (int k = 0; k < rounds; ++k) load += round_cost(k);

    // ---- the rest, cut by the capacities left
    const int32_t idx0 = rounds * ctas;
    int32_t r0 = 0, g0 = 0;
    if (idx0 < n_items) item_at(idx0, by_head, nblocks, hkv, r0, g0);
    const int32_t done = idx0 >= n_items ? cost_all * hkv
                         : by_head       ? g0 * cost_all + before[r0]
                                         : before[r0] * hkv + g0 * cost_of(work_at(r0));
    const int32_t rest = cost_all * hkv - done;
    for (int32_t i = idx0 + tid; i < n_items; i += kPlanThreads) plan.is_cut[i - idx0] = 0;
    const int32_t cap = tid < ctas ? max(0, share - piece_cost - load) : 0;
    const int32_t upto = block_scan(make_int3(cap, 0, 0), warp_sums, total).x;
    if (tid == 0) {
        cut_idx[0] = idx0;
        cut_step[0] = 0;
    }
    if (tid < ctas) {
        // the end of CTA tid's part: position x of the rest (in binary32: only its
        // order counts)
        int32_t idx = n_items, step = 0;
        if (rest > 0 && tid < ctas - 1 && total.x > 0) {
            const int32_t x =
                done + min(rest, int32_t(float(rest) * (float(upto) / float(total.x))));
            int32_t g = 0, y = x;
            if (by_head) {
                g = min(int32_t(uint32_t(x) / uint32_t(cost_all)), hkv - 1);
                y = x - g * cost_all;
            }
            const int32_t times = by_head ? 1 : hkv;
            int lo = 0, hi = nblocks;            // before[lo] <= y / times < before[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (before[mid] * times <= y) lo = mid;
                else hi = mid;
            }
            const int32_t work = work_at(lo);
            const bool halves = few_blocks ? s_work[lo] & 1 : plan.blocks[lo].ntok <= tpt;
            const int32_t steps = halves ? split_steps(work) : work;
            int32_t off = y - before[lo] * times;
            if (!by_head) {
                const int32_t c = cost_of(work);
                g = min(int32_t(uint32_t(off) / uint32_t(c)), hkv - 1);
                off -= g * c;
            }
            idx = by_head ? g * nblocks + lo : lo * hkv + g;
            step = max(off - item_cost, 0) << shift;
            step = min(halves ? split_steps(step) : step, steps);
            if (step < kSnap) step = 0;
            else if (steps - step < kSnap) {
                step = 0;
                ++idx;
            }
            if (idx < idx0) {
                idx = idx0;
                step = 0;
            }
        }
        cut_idx[tid + 1] = idx;
        cut_step[tid + 1] = step;
    }
    __syncthreads();
    int32_t i0 = 0, i1 = 0, s0 = 0, s1 = 0, count = 0, cut = 0;
    if (tid < ctas) {
        i0 = cut_idx[tid];
        s0 = cut_step[tid];
        i1 = cut_idx[tid + 1];
        s1 = cut_step[tid + 1];
        // (a part inside one item may be empty: its zero steps still fill its slot)
        count = i1 - i0 + (s1 > 0);
        // this part begins an item that goes on
        cut = s1 > 0 && (i1 > i0 || s0 == 0);
    }
    const int3 at = block_scan(make_int3(count, cut, 0), warp_sums, total);
    if (tid < ctas) {
        const int32_t p0 = at.x - count;
        plan.piece0[tid] = p0;
        for (int k = 0; k < count; ++k) {
            const int32_t idx = i0 + k, from = k ? 0 : s0;
            int32_t r, g;
            item_at(idx, by_head, nblocks, hkv, r, g);
            Block q = few_blocks ? ordered(r) : plan.blocks[r];
            if (few_blocks) q.prow = s_prow[r];
            const int32_t to = idx == i1 ? s1 : q.steps;
            int32_t prow;
            if (from > 0) prow = tid * plan.slot_rows;
            else if (to < q.steps) prow = (ctas + tid) * plan.slot_rows;
            else prow = q.prow < 0 ? -1 : q.prow + g * 2 * q.ntok * sh.group;
            plan.pieces[p0 + k] = item_of(q, g, from, to, tpt, prow);
            if (from == 0 && to < q.steps) {
                int more = 0;
                while (tid + 1 + more < ctas && cut_idx[tid + 1 + more] == idx &&
                       cut_step[tid + 1 + more] > 0)
                    ++more;
                plan.cuts[at.y - 1] = {r, g, tid, more};
                plan.is_cut[idx - idx0] = 1;
            }
        }
    }
    if (tid == 0) {
        plan.piece0[ctas] = total.x;
        plan.header[kHdrBlocks] = nblocks;
        plan.header[kHdrRounds] = rounds;
        plan.header[kHdrByHead] = by_head;
        plan.header[kHdrSplit] = nsplit;
        plan.header[kHdrCuts] = total.y;
        plan.header[kHdrSplitRows] = s_split_rows;
    }
}

// ------------------------------------------------------------------ the kernel
// Ring positions of an item's tiles, from its first: pair items K0 V0 K1 V1 ..,
// split items KA0 KB0 VA0 VB0 KA1 .. (the last step may have A alone).
struct Order {
    uint32_t base;
    int32_t split, nb;
    __device__ __forceinline__ uint32_t v(int h, int i) const {
        return base + (split ? 4 * i + (i < nb ? 2 + h : 1) : 2 * i + 1);
    }
    __device__ __forceinline__ uint32_t total(int na) const {
        return split ? 2 * (na + nb) : 2 * na;
    }
};

// Bits c < x of the 32 columns from 32 w on.
__device__ __forceinline__ uint32_t below(int32_t x, int w) {
    const int32_t n = min(32, max(0, x - 32 * w));
    return n == 32 ? 0xffffffffu : (1u << n) - 1u;
}

// d = a * b + c on two fp32 pairs.
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
    asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; "
        "fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d; }"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1) {
    asm("{ .reg .b64 a, d; mov.b64 a, {%2, %3}; mov.b64 d, {%0, %1}; "
        "add.rn.f32x2 d, d, a; mov.b64 {%0, %1}, d; }"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
// 32 bytes, a whole sector (in one store where the buffer's alignment allows it).
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8], bool aligned) {
    if (!aligned) {
        uint4 *q = static_cast<uint4 *>(p);
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// Two maxima raised by four scores (two chains in flight).
__device__ __forceinline__ void raise4(float (&mx)[2], const uint32_t *x) {
    mx[0] = max3(mx[0], __uint_as_float(x[0]), __uint_as_float(x[1]));
    mx[1] = max3(mx[1], __uint_as_float(x[2]), __uint_as_float(x[3]));
}
// Makes what follows depend on registers a TMEM load has filled (their values
// are there only after the wait that precedes this).
template <int N>
__device__ __forceinline__ void pin(uint32_t *r) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]),
                          "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}
// Four query elements, scaled below 256 -> their E4M3 codes and those of the rounding
// residuals.  Through fp16, which holds a bf16 number of 2^-14 or more exactly.
__device__ __forceinline__ void e4m3_terms(float p0, float p1, float p2, float p3, uint32_t &t0,
                                           uint32_t &t1) {
    const uint32_t a = pack_f16x2(p0, p1), b = pack_f16x2(p2, p3);
    asm("{ .reg .b16 x, y; .reg .b32 u, v;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 x, %2; cvt.rn.satfinite.e4m3x2.f16x2 y, %3;\n\t"
        "mov.b32 %0, {x, y};\n\t"
        "cvt.rn.f16x2.e4m3x2 u, x; cvt.rn.f16x2.e4m3x2 v, y;\n\t"
        "sub.rn.f16x2 u, %2, u; sub.rn.f16x2 v, %3, v;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 x, u; cvt.rn.satfinite.e4m3x2.f16x2 y, v;\n\t"
        "mov.b32 %1, {x, y}; }"
        : "=&r"(t0), "=r"(t1) : "r"(a), "r"(b));
}

// p = 2^(s sc + neg) of 64 scores: their sums onto `sum`, the pairs rounded to
// bf16 (E4M3 caches: fp16) in t.
template <bool E4>
__device__ __forceinline__ void exponentials(const uint32_t *s, float sc, float neg,
                                             float (&sum)[4], uint32_t (&t)[32]) {
    constexpr int kLag = 2;              // groups between an exponential and its use
    float p[4 * (kLag + 1)];
#pragma unroll
    for (int g = 0; g < 16 + kLag; ++g) {
        if (g < 16) {
            float *x = p + 4 * (g % (kLag + 1));
            fma2(x[0], x[1], __uint_as_float(s[4 * g]), __uint_as_float(s[4 * g + 1]), sc, sc, neg,
                 neg);
            fma2(x[2], x[3], __uint_as_float(s[4 * g + 2]), __uint_as_float(s[4 * g + 3]), sc, sc,
                 neg, neg);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ex2_approx(x[e]);
        }
        if (g >= kLag) {
            const int d = g - kLag;
            const float *x = p + 4 * (d % (kLag + 1));
            add2(sum[0], sum[1], x[0], x[1]);
            add2(sum[2], sum[3], x[2], x[3]);
            t[2 * d] = E4 ? pack_f16x2(x[0], x[1]) : pack_bf16x2(x[0], x[1]);
            t[2 * d + 1] = E4 ? pack_f16x2(x[2], x[3]) : pack_bf16x2(x[2], x[3]);
        }
    }
}

// kWithhold: the test control's form -- no copy is issued, waits are short.
template <int D, bool E4, bool kWithhold>
__global__ void __launch_bounds__(Cfg<D, E4>::kThreads, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
                const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const ChunkArgs a, const Plan plan,
                const Shape sh) {
    using C = Cfg<D, E4>;
    constexpr uint64_t kLimit = kWithhold ? kTestWaitNs : kWaitLimitNs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_addr(base);
    volatile uint32_t *tslot = reinterpret_cast<volatile uint32_t *>(base + kOffSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + kOffFlag);
    auto bar = [&](int i) { return sb + 8u * uint32_t(i); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hkv = a.cache.num_kv_heads, bs = a.cache.block_size;
    const int G = sh.group, tpt = sh.tokens_per_tile;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(kBarFull + s), 1);
            mbar_init(bar(kBarReady + s), 2);
            mbar_init(bar(kBarEmpty + s), E4 ? C::kWideners : 1);
        }
        mbar_init(bar(kBarQFull), E4 ? 256 : 1);
        mbar_init(bar(kBarQEmpty), 1);
        mbar_init(bar(kBarDrain), 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(bar(kBarSFull + h), 1);
            mbar_init(bar(kBarPFull + h), 128);
            mbar_init(bar(kBarPFull + 2 + h), 128);
            mbar_init(bar(kBarPvDone + h), 1);
            mbar_init(bar(kBarP0Done + h), 1);
            mbar_init(bar(kBarOEmpty + h), 128);
            mbar_init(bar(kBarWideFull + h), 32 * C::kWideners);
            mbar_init(bar(kBarWideEmpty + h), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::alloc(sb + kOffSlot, kTmemCols);
        tc::fence_before_sync();
    }
    if (threadIdx.x == kLoadWarp * 32) {
        if (!E4) tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tslot;
    pdl_launch_dependents();
    pdl_wait();
    const int rounds = plan.header[kHdrRounds], piece0 = plan.piece0[blockIdx.x];
    const int num_items = rounds + plan.piece0[blockIdx.x + 1] - piece0;
    // this CTA's item `it`: whole ones first, then its pieces
    auto read_item = [&](int it) {
        Item r;
        if (it >= rounds) {
            const int4 *p = reinterpret_cast<const int4 *>(plan.pieces + piece0 + it - rounds);
            int4 *d = reinterpret_cast<int4 *>(&r);
            d[0] = p[0];
            d[1] = p[1];
            d[2] = p[2];
        } else {
            int32_t blk, g;
            item_at(round_item(it, blockIdx.x, plan.ctas), plan.header[kHdrByHead] != 0,
                    plan.header[kHdrBlocks], hkv, blk, g);
            Block q;
            const int4 *p = reinterpret_cast<const int4 *>(plan.blocks + blk);
            int4 *d = reinterpret_cast<int4 *>(&q);
            d[0] = p[0];
            d[1] = p[1];
            r = item_of(q, g, 0, q.steps, tpt, q.prow < 0 ? -1 : q.prow + g * 2 * q.ntok * G);
        }
        return r;
    };

    if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == kLoadWarp) {
        // ------------------------------------------------------------ producer
        const int box = min(bs, kKeys);
        const int nbox = kKeys / box, log_bs = 31 - __clz(bs);
        uint32_t ring = 0, items_done = 0;
        uint32_t armed = 0, armed_parity = 0;
        uint32_t q_armed = 0, q_parity = 0;
        bool ok = !kWithhold;
        for (int it = 0; it < num_items && ok; ++it) {
            const Item r = read_item(it);
            if (r.na == 0) continue;
            const int g = r.g;
            const Tiles tl = tiles_of(r.pos, r.ntok, a.window, a.sinks);
            const int32_t pmax = r.pos + r.ntok - 1;
            const int32_t *table = a.block_tables + int64_t(r.b) * a.max_blocks;
            // This lane's box of step i -- of a pair item lanes 0 .. nbox - 1, of a split
            // item half A's in lanes 0 .. 15 and half B's in 16 .. 31 -- as its first
            // key, or -1: nothing to copy.
            auto key_of = [&](int i) -> int32_t {
                const int bx = r.split ? lane & 15 : lane, half = r.split ? lane >> 4 : 0;
                if (bx >= nbox || i >= (half ? r.nb : r.na)) return -1;
                const int v = r.v0 + (half ? r.na : 0) + i;
                const int32_t key = (v < tl.sink_tiles ? v : v + tl.gap) * kKeys + bx * box;
                return key > pmax || (key + box - 1 < tl.lo && key >= a.sinks) ? -1 : key;
            };
            // The entry of its block, and the pool row that entry stands for (two
            // functions, a step apart: the first one's load need not be waited for).
            auto entry_of = [&](int i) -> int32_t {
                const int32_t key = key_of(i);
                return key < 0 ? 0 : table[key >> log_bs];
            };
            auto row_of = [&](int i, int32_t phys) -> int32_t {
                const int32_t key = key_of(i);
                if (key < 0) return -1;
                if (phys < 0 || phys >= a.cache.num_blocks) {
                    raise_status(a.status, PKV_DEV_BLOCK_ID);
                    return g * bs;                  // some block's rows stand in
                }
                return (phys * hkv + g) * bs + (key & (bs - 1));
            };
            auto load = [&](const CUtensorMap *map, int32_t y) -> bool {
                const uint32_t stage = ring % C::kStages, phase = (ring / C::kStages) & 1u;
                if (!__all_sync(0xffffffffu, pipe_wait(bar(kBarEmpty + stage), phase ^ 1u,
                                                       a.status, abort_flag, kLimit)))
                    return false;
                const uint32_t live = __ballot_sync(0xffffffffu, y >= 0);
                if (lane == 0) {
                    if (E4 && map == &tmap_k)
                        for (int k = 1; k < C::kWideners; ++k) mbar_arrive(bar(kBarEmpty + stage));
                    mbar_arrive_expect_tx(bar(kBarFull + stage),
                                          __popc(live) * uint32_t(box) * D * C::kElem);
                }
                armed |= 1u << stage;
                armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                __syncwarp();
                if (y >= 0) {
                    const uint32_t dst = sb + C::kOffRing + stage * C::kStage +
                                         uint32_t(lane * box) * D * C::kElem;
                    if constexpr (D * C::kElem == 256)
                        tma_load_4d(dst, map, 0, 0, 0, y >> 3, bar(kBarFull + stage));
                    else
                        tma_load_2d(dst, map, 0, y, bar(kBarFull + stage));
                }
                ++ring;
                return true;
            };
            // the item's query tiles, once the last item's are no longer read
            auto load_q = [&]() -> bool {
                if constexpr (!E4) {
                    if (!__all_sync(0xffffffffu,
                                    pipe_wait(bar(kBarQEmpty), (items_done & 1u) ^ 1u, a.status,
                                              abort_flag, kLimit)))
                        return false;
                    if (lane == 0) {
                        const int tiles = r.split ? 1 : 2;
                        mbar_arrive_expect_tx(bar(kBarQFull), tiles * uint32_t(tpt * G) * D * 2);
                        for (int t = 0; t < tiles; ++t)
                            for (int half = 0; half < D / 64; ++half)
                                tma_load_3d(sb + C::kOffQ + t * C::kQTile + half * C::kHalfTile,
                                            &tmap_q, half * 64, g * G, r.qrow + t * tpt,
                                            bar(kBarQFull));
                    }
                    __syncwarp();
                    q_armed = 1;
                    q_parity = items_done & 1u;
                }
                ++items_done;
                return true;
            };
            // Rows are known kAhead steps before their copy, so that the copies wait for
            // no table; the queries' buffer frees late, so the item's first keys go
            // before them.  (Copies to L2 ahead of the ring's made split items slower:
            // single tokens under a window of 4,096 228 -> 297 us.)
            constexpr int kAhead = 3;
            int32_t y[kAhead], phys[kAhead + 1];
#pragma unroll
            for (int k = 0; k <= kAhead; ++k) phys[k] = entry_of(k);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) y[k] = row_of(k, phys[k]);
            int32_t pending = phys[kAhead];
            for (int i = 0; i < r.na && ok; ++i) {
                if (!r.split) {
                    ok = load(&tmap_k, y[0]) && (i > 0 || load_q()) && load(&tmap_v, y[0]);
                } else {
                    const int32_t yb = __shfl_down_sync(0xffffffffu, y[0], 16);
                    const int32_t y0 = lane < 16 ? y[0] : -1, y1 = lane < 16 ? yb : -1;
                    const bool both = i < r.nb;
                    ok = load(&tmap_k, y0) && (!both || load(&tmap_k, y1)) &&
                         (i > 0 || load_q()) && load(&tmap_v, y0) && (!both || load(&tmap_v, y1));
                }
#pragma unroll
                for (int k = 0; k + 1 < kAhead; ++k) y[k] = y[k + 1];
                y[kAhead - 1] = row_of(i + kAhead, pending);
                pending = entry_of(i + kAhead + 1);
            }
        }
        // Do not leave while copies may still land in this CTA's shared memory.
        if (lane == 0) {
            for (int s = 0; s < C::kStages; ++s)
                if (armed & (1u << s))
                    mbar_wait(bar(kBarFull + s), (armed_parity >> s) & 1u, a.status, kLimit);
            if (q_armed) mbar_wait(bar(kBarQFull), q_parity, a.status, kLimit);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMA issuer
        // One thread issues blocks of [value product of step i, score product of
        // step i + 1], half A's and half B's in turn, so that one half's softmax
        // runs under the other's products.  What the thread does between two
        // products leaves the tensor cores idle, so it does little: ring positions
        // are counted, not divided, and nothing is kept that spills.
        if (tc::elect_one()) {
            uint32_t slot = 0, lap = 0;          // ring position: stage and lap parity
            uint32_t item_bit = 0;               // items done, mod 2
            uint32_t np[2] = {0, 0};             // tiles whose probabilities were taken, mod 2
            uint32_t nitem[2] = {0, 0};          // items begun, by half, mod 2
            uint32_t wide = 0, wide_lap = 0;     // next buffer of widened values (E4M3)
            bool ok = true;
            auto wait = [&](uint32_t b, uint32_t parity) {
                return pipe_wait(b, parity, a.status, abort_flag, kLimit);
            };
            // the ring entry `off` positions on: its stage, waited for
            auto entry = [&](uint32_t off, uint32_t &stage) {
                stage = slot + off;
                uint32_t l = lap;
                if (stage >= C::kStages) {
                    stage -= C::kStages;
                    l ^= 1u;
                }
                return wait(bar(C::kTended ? kBarReady : kBarFull) + 8u * stage, l);
            };
            auto advance = [&](uint32_t n) {
                slot += n;
                if (slot >= C::kStages) {
                    slot -= C::kStages;
                    lap ^= 1u;
                }
            };
            auto scores = [&](int h, bool second_q, uint32_t stage) {
                const uint32_t ds = tmem + kKeys * h;
                const uint32_t kb = sb + C::kOffRing + stage * C::kStage;
                const uint64_t kd = tc::smem_desc(kb, 16, D * C::kElem == 256 ? 2048 : 1024);
                const uint64_t q =
                    tc::smem_desc(sb + C::kOffQ + (second_q ? C::kQTile : 0u), 16, 1024);
                if constexpr (E4) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_e4m3(ds, q + ((t * C::kHalfTile + 32 * kk) >> 4),
                                         kd + ((32 * kk) >> 4), C::kIdS, (t | kk) != 0);
                } else {
#pragma unroll
                    for (int half = 0; half < D / 64; ++half)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc::mma_bf16(ds, q + ((half * C::kHalfTile + 32 * kk) >> 4),
                                         kd + ((half * 1024 + 32 * kk) >> 4), C::kIdS,
                                         (half | kk) != 0);
                }
                tc::commit(bar(kBarSFull + h));
            };
            // part 0 or 1 (64 keys) of a value product; `first`: O begins
            auto values = [&](int h, bool first, uint32_t stage, int part) {
                const uint32_t dO = tmem + kColO + 128 * h, p = tmem + kKeys * h;
                const uint32_t vb = sb + (E4 ? C::kOffWide + stage * C::kWide
                                             : C::kOffRing + stage * C::kStage);
                const uint64_t vd = D == 128 ? tc::smem_desc(vb, 1024, 2048)
                                             : tc::smem_desc(vb, 16384, 1024);
#pragma unroll
                for (int kk = 4 * part; kk < 4 * part + 4; ++kk)
                    tc::mma_bf16_ts(dO, p + 8 * kk, vd + (((D == 128 ? 4096 : 2048) * kk) >> 4),
                                    C::kIdO, kk || !first);
            };
            for (int it = 0; it < num_items && ok; ++it) {
                const Item r = read_item(it);
                if (r.na == 0) continue;
                const int na = r.na, nb = r.nb;
                const bool split = r.split;
                if (!(ok = wait(bar(kBarQFull), item_bit))) break;
                item_bit ^= 1u;
                uint32_t st;
                // ---- the first scores
                if (!(ok = entry(0, st))) break;
                tc::fence_after_sync();
                scores(0, false, st);
                if (split) tc::commit(bar(kBarEmpty) + 8u * st);
                if (nb > 0) {
                    if (split && !(ok = entry(1, st))) break;
                    tc::fence_after_sync();
                    scores(1, !split, st);
                    tc::commit(bar(kBarEmpty) + 8u * st);
                }
                if (na == 1) tc::commit(bar(kBarQEmpty));
                // entries of step 0 from here: pair items V0 K1, split items VA0 VB0 KA1 KB1
                advance(split && nb > 0 ? 2 : 1);
                for (int i = 0; i < na && ok; ++i) {
                    const bool more = i + 1 < na;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h && i >= nb) continue;
                        const bool scores_too = h ? i + 1 < nb : more;
                        uint32_t vs = 0, ks = 0;
                        // (half B of a pair item: its tiles are A's, waited for there)
                        if (h == 0 || split) {
                            const bool both = split && i < nb;
                            ok = E4 ? wait(bar(kBarWideFull) + 8u * wide, wide_lap)
                                    : entry(both ? h : 0, vs);
                            if (ok && scores_too) ok = entry(both ? 2 + h : 1, ks);
                        } else {
                            vs = slot;
                            ks = slot + 1 == C::kStages ? 0 : slot + 1;
                        }
                        if (E4) vs = wide;
                        auto next_scores = [&] {
                            if (!scores_too) return;
                            scores(h, h && !split, ks);
                            if (split || h) tc::commit(bar(kBarEmpty) + 8u * ks);
                        };
                        if (!ok) break;
                        if (i == 0) {
                            ok = wait(bar(kBarOEmpty + h), nitem[h] ^ 1u);
                            nitem[h] ^= 1u;
                            if (!ok) break;
                        }
                        const uint32_t pf = bar(kBarPFull) + 8u * h;
                        const uint32_t pp = np[h];
                        if (!(ok = wait(pf, pp))) break;
                        tc::fence_after_sync();
                        // the first 64 keys' product while the others' softmax goes on
                        values(h, i == 0, vs, 0);
                        tc::commit(bar(kBarP0Done + h));
                        if (!(ok = wait(pf + 16u, pp))) break;
                        tc::fence_after_sync();
                        values(h, i == 0, vs, 1);
                        np[h] ^= 1u;
                        next_scores();
                        // (the other value products' end is told with the next scores')
                        if (!scores_too) tc::commit(bar(kBarPvDone + h));
                        if (split || h) {
                            tc::commit(bar(E4 ? kBarWideEmpty : kBarEmpty) + 8u * vs);
                            wide_lap ^= wide;
                            wide ^= 1u;
                        }
                    }
                    // the item's last score product frees its queries
                    if (i + 2 == na) tc::commit(bar(kBarQEmpty));
                    advance(split ? (i < nb ? 2 : 1) + (more ? 1 : 0) + (i + 1 < nb ? 1 : 0)
                                  : 1 + (more ? 1 : 0));
                }
            }
            tc::commit(bar(kBarDrain));
            mbar_wait(bar(kBarDrain), 0, a.status, kLimit);
        }
        __syncwarp();
    } else if (C::kTended) {
        // ------------------------------------- value rows no row of the item sees
        // Warps 10 and 11, 64 keys each: such rows become 0 before the value product
        // reads them.  Every tile of the ring passes here, keys too: copies may land in
        // another order than they were issued in, and a role that waited for some
        // phases of a stage only could take one for the next.
        uint32_t stage = 0, lap = 0;
        bool ok = true;
        for (int it = 0; it < num_items && ok; ++it) {
            const Item r = read_item(it);
            if (r.na == 0) continue;
            const Tiles tl = tiles_of(r.pos, r.ntok, a.window, a.sinks);
            const int32_t pmax = r.pos + r.ntok - 1;
            const int total = r.split ? 2 * (r.na + r.nb) : 2 * r.na;
            for (int e = 0; e < total; ++e) {
                // entries K0 V0 K1 .., or KA0 KB0 VA0 VB0 KA1 .. KA VA
                int v = -1;
                if (!r.split) {
                    if (e & 1) v = e >> 1;
                } else if (e < 4 * r.nb) {
                    if (e & 2) v = (e & 1 ? r.na : 0) + (e >> 2);
                } else if (e & 1) {
                    v = r.nb;
                }
                ok = __all_sync(0xffffffffu,
                                pipe_wait(bar(kBarFull) + 8u * stage, lap, a.status, abort_flag,
                                          kLimit));
                if (!ok) break;
                if (v >= 0) {
                    v += r.v0;
                    const int32_t k0 = (v < tl.sink_tiles ? v : v + tl.gap) * kKeys;
                    if (k0 + kKeys - 1 > pmax ||
                        (k0 < tl.lo && max(k0, a.sinks) < min(tl.lo, k0 + kKeys))) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int row = (warp - kLoadWarp - 1) * 64 + 32 * u + lane;
                            const int32_t key = k0 + row;
                            if (key > pmax || (key < tl.lo && key >= a.sinks)) {
                                uint4 *d = reinterpret_cast<uint4 *>(
                                    base + C::kOffRing + stage * C::kStage + row * 128);
#pragma unroll
                                for (int c = 0; c < 8; ++c) d[c] = make_uint4(0, 0, 0, 0);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (lane == 0) mbar_arrive(bar(kBarReady) + 8u * stage);
                if (++stage == C::kStages) {
                    stage = 0;
                    lap ^= 1u;
                }
            }
        }
    } else if (E4 && warp >= kWidenWarp) {
        // ------------------------------------------------- values widened to fp16
        // Every code is an fp16 number.  Eight lanes take a key's 128 codes (16
        // each, the chunks of a row in turn: no bank twice), a pass 8 keys; keys that
        // no row of the item sees become 0.
        uint32_t ring = 0, wide = 0, lap = 1;
        bool ok = true;
        const int c = lane & 7, r0 = (warp & 1) * 4 + (lane >> 3), hi8 = (warp >> 1) & 1;
        const uint32_t from = uint32_t(r0 * 128 + ((c ^ r0) << 4));
        const int half = c >> 2, chunk = (c & 3) * 2;
        const uint32_t to0 = uint32_t(half * 1024 + r0 * 128 + (((chunk + half) ^ r0) << 4));
        const uint32_t to1 = uint32_t(half * 1024 + r0 * 128 + (((chunk + 1 - half) ^ r0) << 4));
        for (int it = 0; it < num_items && ok; ++it) {
            const Item r = read_item(it);
            if (r.na == 0) continue;
            const Tiles tl = tiles_of(r.pos, r.ntok, a.window, a.sinks);
            const int32_t pmax = r.pos + r.ntok - 1;
            const Order ord{ring, r.split, r.nb};
            for (int j = 0; j < r.na + (r.split ? r.nb : 0) && ok; ++j) {
                const int h = r.split ? (j < 2 * r.nb ? j & 1 : 0) : 0;
                const int i = r.split ? (j < 2 * r.nb ? j >> 1 : r.na - 1) : j;
                const int v = r.v0 + (h ? r.na : 0) + i;
                const uint32_t vp = ord.v(h, i), stage = vp % C::kStages;
                // (The buffer first: its last product came after every wait for the key
                // tile that was in this stage before.  Copies may land in another order
                // than they were issued in; without that this wait could take the key
                // tile's phase for this one's.)
                ok = __all_sync(0xffffffffu,
                                pipe_wait(bar(kBarWideEmpty + wide), lap, a.status, abort_flag,
                                          kLimit) &&
                                    pipe_wait(bar(kBarFull + stage), (vp / C::kStages) & 1u,
                                              a.status, abort_flag, kLimit));
                if (!ok) break;
                const uint8_t *src = base + C::kOffRing + stage * C::kStage + from + hi8 * 8192;
                uint8_t *dst = base + C::kOffWide + wide * C::kWide + hi8 * 16384;
                const int32_t k0 = (v < tl.sink_tiles ? v : v + tl.gap) * kKeys;
                const bool some = k0 + kKeys - 1 > pmax ||
                                  (k0 < tl.lo && max(k0, a.sinks) < min(tl.lo, k0 + kKeys));
                // four keys' chunks are fetched before the last four are written
                uint4 x[2][4];
                auto fetch = [&](int q) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[q & 1][e] =
                            *reinterpret_cast<const uint4 *>(src + (4 * q + e) * 1024);
                };
                fetch(0);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (q < 1) fetch(q + 1);
                    uint4 (&y)[4] = x[q & 1];
                    if (some) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int32_t key = k0 + r0 + 64 * hi8 + 8 * (4 * q + e);
                            if (key > pmax || (key < tl.lo && key >= a.sinks))
                                y[e] = make_uint4(0, 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint2 a0 = e4m3x4_to_f16x4(y[e].x), a1 = e4m3x4_to_f16x4(y[e].y);
                        const uint2 b0 = e4m3x4_to_f16x4(y[e].z), b1 = e4m3x4_to_f16x4(y[e].w);
                        const uint4 lo = make_uint4(a0.x, a0.y, a1.x, a1.y);
                        const uint4 hi = make_uint4(b0.x, b0.y, b1.x, b1.y);
                        uint8_t *d = dst + (4 * q + e) * 2048;
                        *reinterpret_cast<uint4 *>(d + to0) = half ? hi : lo;
                        *reinterpret_cast<uint4 *>(d + to1) = half ? lo : hi;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(kBarWideFull + wide));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kBarEmpty + stage));
                lap ^= wide;
                wide ^= 1u;
            }
            ring += ord.total(r.na);
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        // -------------------------------------------- softmax and epilogue
        // A thread whose wait gave up arrives once more for its tile's phases at most, and
        // for none after them: its warp takes no further tiles (kEndsItem), or goes through
        // them without arriving.  Arrivals ahead would stand for those of rows that are
        // behind, which the tensor cores would then read unwritten, and more than a phase
        // has pending are a fault.  So no product is issued past it, the others' waits give
        // up too, and what rows the CTA has not finished become NaN.
        const int h = warp >> 2;                         // half
        const int row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + kKeys * h + lanes;    // S, P
        const uint32_t to = tmem + kColO + 128 * h + lanes;
        const int tok_row = row / G, head_row = row - tok_row * G;
        const bool out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
        uint32_t ring = 0, np = 0, nitem = 0, items_done = 0;
        uint32_t s_par = 0;
        bool ok = true;
        for (int it = 0; it < num_items; ++it) {
            const Item r = read_item(it);
            const int g = r.g;
            const int n = h ? r.nb : r.na;
            const int tok0 = r.split ? 0 : h * tpt;      // the half's first token
            float sc = a.scale * kLog2e;
            float m = -INFINITY, l = 0.f;            // reference, sum against it
            const bool has_row = tok_row < tpt && tok0 + tok_row < r.ntok;
            if (!has_row) sc = m = 0.f;              // any bits
            if constexpr (E4) {
                sc *= a.k_scale[g];
                if (r.na > 0) {
                    // this half's query rows as two E4M3 terms, scaled by a power
                    // of two that puts the row's largest element in [128, 256)
                    ok = ok && pipe_wait(bar(kBarQEmpty), (items_done & 1u) ^ 1u, a.status,
                                         abort_flag, kLimit);
                    const uint4 *src = static_cast<const uint4 *>(a.q) +
                        (int64_t(r.qrow + min(tok0 + tok_row, r.ntok - 1)) * a.num_q_heads + g * G +
                         head_row) * (D / 8);
                    float big = 0.f;
                    bool finite = true;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 x = src[i];
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = fabsf(bf16_lo_to_f32(w[e]));
                            const float v = fabsf(bf16_hi_to_f32(w[e]));
                            finite = finite && u < INFINITY && v < INFINITY;
                            big = fmaxf(big, fmaxf(u, v));
                        }
                    }
                    // big = 1.f 2^e: 2^(7 - e), within the normal range
                    const int e = min(126, max(-118, int(__float_as_uint(big) >> 23) - 127));
                    const float up = __uint_as_float(uint32_t(134 - e) << 23);
                    sc *= __uint_as_float(uint32_t(120 + e) << 23);
                    // Masked scores are -inf, and -inf * 0 a NaN: rows of zeros or of the
                    // smallest numbers over a small key scale must not lose sc.  (Scores
                    // stay below 2^25, so at the smallest normal number all are 0.)
                    if (sc < 1.17549435e-38f) sc = 1.17549435e-38f;
                    if (!finite) sc = __int_as_float(0x7fc00000);       // inf or NaN: a NaN row
                    if (ok && (h == 0 || !r.split)) {
                        uint8_t *q0 = base + C::kOffQ + h * C::kQTile + row * 128;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            const uint4 x0 = src[2 * i], x1 = src[2 * i + 1];
                            const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                            uint32_t t0[4], t1[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                e4m3_terms(bf16_lo_to_f32(w[2 * k]) * up,
                                           bf16_hi_to_f32(w[2 * k]) * up,
                                           bf16_lo_to_f32(w[2 * k + 1]) * up,
                                           bf16_hi_to_f32(w[2 * k + 1]) * up, t0[k], t1[k]);
                            const int off = ((i ^ row) & 7) << 4;
                            *reinterpret_cast<uint4 *>(q0 + off) =
                                make_uint4(t0[0], t0[1], t0[2], t0[3]);
                            *reinterpret_cast<uint4 *>(q0 + C::kHalfTile + off) =
                                make_uint4(t1[0], t1[1], t1[2], t1[3]);
                        }
                        fence_proxy_async_smem();
                    }
                    if (ok) mbar_arrive(bar(kBarQFull));
                }
            }
            if (r.na > 0) ++items_done;
            const int v0 = r.v0 + (r.split && h ? r.na : 0);
            const Tiles tl = tiles_of(r.pos, r.ntok, a.window, a.sinks);
            const int32_t pmax = r.pos + r.ntok - 1, pos = r.pos + tok0 + tok_row;
            // positions of the warp's rows (none: the largest below the smallest)
            const int32_t first = __reduce_min_sync(0xffffffffu, has_row ? pos : INT_MAX);
            const int32_t last = __reduce_max_sync(0xffffffffu, has_row ? pos : INT_MIN);
            // Virtual tiles [clear0, clear1): each of them sees every key.
            const int clear0 =
                max((a.window > 0 && last >= a.window ? (last - a.window) / kKeys + 1 : 0) - tl.gap,
                    tl.sink_tiles);
            const int clear1 = (first == INT_MAX ? 0 : max(first + 1, 0) / kKeys) - tl.gap;
            const Order ord{ring, r.split, r.nb};
            for (int i = 0; i < n; ++i) {
                const int v = v0 + i;
                const bool clear = v >= clear0 && v < clear1;
                const int32_t tile_key = (v < tl.sink_tiles ? v : v + tl.gap) * kKeys;
                ok = ok && pipe_wait(bar(kBarSFull + h), s_par, a.status, abort_flag, kLimit);
                if constexpr (C::kEndsItem) {
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                } else {
                    __syncwarp();
                }
                tc::fence_after_sync();
                // ---- value rows no row of the item sees: zeroed, thread = key.  (These
                // scores came after every wait for the tile that was in the stage
                // before, so the wait cannot take that tile's phase for this one's.)
                if (!C::kTended && !E4 && !clear) {
                    const int32_t key = tile_key + row;
                    const bool unseen = key > pmax || (key < tl.lo && key >= a.sinks);
                    if (__any_sync(0xffffffffu, unseen)) {
                        const uint32_t vp = ord.v(h, i), stage = vp % C::kStages;
                        ok = ok && pipe_wait(bar(kBarFull + stage), (vp / C::kStages) & 1u,
                                             a.status, abort_flag, kLimit);
                        if (ok && unseen) {
                            uint8_t *vt = base + C::kOffRing + stage * C::kStage;
                            vt += (row >> 3) * 2048 + (row & 7) * 128;
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4 *>(vt + (c >> 3) * 1024 + (c & 7) * 16) =
                                    make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                // ---- probabilities, rounded to 16 bits over S's columns, 64 keys at a
                // time, against the row's reference m.  m need not be the maximum: a
                // number with a full exponent (bf16's) holds 2^(score - m) as exactly
                // whatever m is, short of overflow; for fp16 they are lifted as far as
                // its range allows.  So they are taken against the first maximum,
                // and the reference rises only when the sum of a row's 64 passes kMost;
                // they are then taken again.  A loop, not unrolled: the code of one part
                // stays in the instruction cache beside the issuing thread's.
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    uint32_t x[64], t[32];
                    const int32_t k0 = tile_key + 64 * part;
                    // no row of the warp sees any of the keys: nothing is computed
                    if (!clear &&
                        (k0 > last ||
                         (a.window > 0 && k0 + 63 <= first - a.window && k0 >= a.sinks))) {
                        if (last != INT_MIN) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) t[j] = 0u;
                            tc::st32(ts + 32 * part, t);
                            tc::wait_st();
                            tc::fence_before_sync();
                        }
                        if (C::kEndsItem || ok) mbar_arrive(bar(kBarPFull + 2 * part + h));
                        continue;
                    }
                    tc::ld32(ts + 64 * part, x);
                    tc::ld32(ts + 64 * part + 32, x + 32);
                    tc::wait_ld();
                    pin<32>(x);
                    pin<32>(x + 32);
                    // unless every row of the warp sees all of them
                    if (!clear &&
                        (k0 + 63 > first ||
                         (a.window > 0 && k0 <= last - a.window && k0 + 63 >= a.sinks))) {
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            uint32_t see = pos >= 0 ? below(pos - k0 + 1, w) : 0u;
                            if (a.window > 0)
                                see &= ~below(pos - k0 - a.window + 1, w) | below(a.sinks - k0, w);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((see >> j) & 1u)) x[32 * w + j] = 0xff800000u;
                        }
                    }
                    float total;
                    for (bool again = false;; again = true) {
                        float neg;
                        if constexpr (E4) neg = m == -INFINITY ? 0.f : fmaf(-m, sc, kLift);
                        else neg = m == -INFINITY ? 0.f : -m * sc;
                        float sum[4] = {0.f, 0.f, 0.f, 0.f};
                        exponentials<E4>(x, sc, neg, sum, t);
                        total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        const bool rise = total > C::kMost || m == -INFINITY;
                        if (!__any_sync(0xffffffffu, rise && !again)) break;
                        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int j = 0; j < 64; j += 4) raise4(mx, x + j);
                        // (a row that need not rise keeps m and, to the bit, its terms:
                        // what a row gives does not depend on its neighbours)
                        const float mn = rise ? fmaxf(m, fmaxf(mx[0], mx[1])) : m;
                        const float f = m == -INFINITY ? 0.f : ex2_approx((m - mn) * sc);
                        if (part || i > 0) {
                            // rescale.  These scores were told after the last tile's value
                            // product; that of this tile's first keys has to be waited for.
                            if (part)
                                ok = ok && pipe_wait(bar(kBarP0Done + h), np & 1u, a.status,
                                                     abort_flag, kLimit);
                            __syncwarp();
                            tc::fence_after_sync();
#pragma unroll
                            for (int j = 0; j < D; j += 16) {
                                uint32_t o[16];
                                tc::ld16(to + j, o);
                                tc::wait_ld();
                                pin<16>(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tc::st16(to + j, o);
                            }
                        }
                        l *= f;
                        m = mn;
                    }
                    __syncwarp();
                    tc::st32(ts + 32 * part, t);
                    tc::wait_st();
                    tc::fence_before_sync();
                    if (C::kEndsItem || ok) mbar_arrive(bar(kBarPFull + 2 * part + h));
                    l += total;
                }
                ++np;
                s_par ^= 1u;
            }

            // ---- epilogue
            if (n > 0) {
                ok = ok && pipe_wait(bar(kBarPvDone + h), nitem & 1u, a.status, abort_flag,
                                     kLimit);
                ++nitem;
                __syncwarp();
                tc::fence_after_sync();
            }
            ok = __all_sync(0xffffffffu, ok);
            const float nan = __int_as_float(0x7fc00000);
            float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            if constexpr (E4) inv *= a.v_scale[g];
            float lse = l > 0.f || l != l ? (m * sc + log2f(l)) * kLn2 : -INFINITY;
            if constexpr (E4) lse -= kLift * kLn2;
            if (!ok) inv = lse = nan;
            ring += ord.total(r.na);
            const int tok = (r.split ? 0 : h * tpt) + tok_row;
            const bool live = tok_row < tpt && tok < r.ntok;
            const bool direct = r.prow < 0;
            const int64_t orow = int64_t(r.qrow + tok) * a.num_q_heads + g * G + head_row;
            const int64_t prow = int64_t(r.prow) + (r.split ? h * r.ntok * G : 0) + tok * G + head_row;
            // half B of a split item without a tile of its own adds nothing to a direct row
            const bool writes = live && !(direct && r.split && h == 1);
            // All of the row into registers, by converged warps, before the rows
            // part ways (the warp-wide loads are only defined for a whole warp).
            uint32_t o[D];
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < D; j += 32) tc::ld32(to + j, o + j);
                tc::wait_ld();
#pragma unroll
                for (int j = 0; j < D; j += 32) pin<32>(o + j);
                tc::fence_before_sync();
                if (ok) mbar_arrive(bar(kBarOEmpty + h));
            } else {
#pragma unroll
                for (int e = 0; e < D; ++e) o[e] = 0u;
            }
            if (writes && direct) {
                uint16_t *dst = static_cast<uint16_t *>(a.out) + orow * D;
#pragma unroll
                for (int e = 0; e < D; e += 16) {
                    uint32_t w[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        w[x] = pack_bf16x2(__uint_as_float(o[e + 2 * x]) * inv,
                                           __uint_as_float(o[e + 2 * x + 1]) * inv);
                    store32(dst + e, w, out32);
                }
            } else if (writes) {
                float *dst = plan.o_part + prow * D;
#pragma unroll
                for (int e = 0; e < D; e += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        w[x] = __float_as_uint(__uint_as_float(o[e + x]) * inv);
                    store32(dst + e, w, true);
                }
            }
            if (writes) {
                if (!direct) plan.lse_part[prow] = lse;
                else if (a.lse) a.lse[orow] = lse;
            }
        }
    }

    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------- the merge
// D / 4 lanes a row: out = sum_c e^{lse_c - M} o_c / sum_c e^{lse_c - M}
// over the row's partials, each already divided by its own sum.  A NaN partial
// makes the row NaN; empty ones (lse = -inf) weigh nothing.
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 4;            // rows of a warp's unit of work (each row waits for
                                         // its partials: 16 rows a warp 23 us, 4 rows 9, of
                                         // a ragged batch of 24)

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
chunk_merge_kernel(const ChunkArgs a, const Plan plan, const Shape sh) {
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;
    pdl_wait();
    pdl_launch_dependents();
    const int hkv = a.cache.num_kv_heads, G = sh.group;
    // the split items taken whole (two partials of at most kRows rows each), then the cuts
    constexpr int kUnits = 2 * kRows / kMergeRows;
    const int32_t n_short = plan.header[kHdrSplit] * hkv;
    const int32_t n_half =
        n_short * ((plan.header[kHdrSplitRows] + kMergeRows - 1) / kMergeRows);
    const int32_t total = n_half + plan.header[kHdrCuts] * kUnits;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, c = lane % kLanes;
    const int nblocks = plan.header[kHdrBlocks];
    const int32_t idx0 = plan.header[kHdrRounds] * plan.ctas;
    const float4 *op = reinterpret_cast<const float4 *>(plan.o_part) + c;
    constexpr int kWarps = kMergeThreads / 32;
    for (int32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5); w < total; w += gridDim.x * kWarps) {
        int blk, g, row0, count, halves = 2;
        int64_t first, next;                 // rows of the first piece, and of the others'
        if (w < n_half) {
            // (unit-major, so that the units past a short item's rows end up in other warps)
            const int32_t unit = w / n_short, sg = w - unit * n_short;
            row0 = unit * kMergeRows;
            blk = plan.split[sg / hkv];
            g = sg % hkv;
            count = 2;
            first = next = 0;
        } else {
            const Cut cut = plan.cuts[(w - n_half) / kUnits];
            blk = cut.block;
            g = cut.g;
            row0 = (w - n_half) % kUnits * kMergeRows;
            count = 1 + cut.more;
            first = int64_t(plan.ctas + cut.cta) * plan.slot_rows;
            next = int64_t(cut.cta) * plan.slot_rows;
        }
        const Block m = plan.blocks[blk];
        const int rows = m.ntok * G;
        if (row0 >= rows) continue;
        if (w < n_half) {
            const int32_t idx = plan.header[kHdrByHead] ? g * nblocks + blk : blk * hkv + g;
            if (idx >= idx0 && plan.is_cut[idx - idx0]) continue;
            first = next = m.prow + int64_t(g) * 2 * rows;
        } else {
            halves = m.ntok <= sh.tokens_per_tile ? 2 : 1;
            count *= halves;
        }
        const int end = min(rows, row0 + kMergeRows);
#pragma unroll 2
        for (int row = row0 + sub; row < end; row += kAtOnce) {
            // partial p: piece p / halves, half p % halves
            auto at = [&](int p) {
                const int piece = halves == 2 ? p >> 1 : p;
                return (piece ? next + int64_t(piece) * plan.slot_rows : first) +
                       (halves == 2 ? (p & 1) * rows : 0) + row;
            };
            float M = -INFINITY, W = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            bool broken = false;
            for (int p0 = 0; p0 < count; p0 += 4) {
                float l[4];
                float4 x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool in = p0 + u < count;
                    const int64_t r = in ? at(p0 + u) : 0;
                    l[u] = in ? plan.lse_part[r] : -INFINITY;
                    x[u] = in ? op[r * kLanes] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float mc = M;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    broken |= l[u] != l[u];
                    mc = fmaxf(mc, l[u]);
                }
                if (mc == -INFINITY) continue;
                const float f = expf(M - mc);
                W *= f;
                acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float wt = expf(l[u] - mc);
                    if (wt != 0.f) {
                        W += wt;
                        acc.x = fmaf(wt, x[u].x, acc.x); acc.y = fmaf(wt, x[u].y, acc.y);
                        acc.z = fmaf(wt, x[u].z, acc.z); acc.w = fmaf(wt, x[u].w, acc.w);
                    }
                }
                M = mc;
            }
            const int64_t orow = (int64_t(m.qrow) + row / G) * a.num_q_heads + g * G + row % G;
            float inv = W > 0.f ? 1.f / W : 0.f;
            float lse = W > 0.f ? M + logf(W) : -INFINITY;
            if (broken) inv = lse = __int_as_float(0x7fc00000);
            reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + orow * D)[c] = make_uint2(
                pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (c == 0 && a.lse) a.lse[orow] = lse;
        }
    }
}

// ------------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 chunk_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

bool encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *at,
            const cuuint64_t *dim, const cuuint64_t *stride, const cuuint32_t *box) {
    auto fn = chunk_encode_fn();
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn && fn(map, type, cuuint32_t(rank), const_cast<void *>(at), dim, stride, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool as rows of D elements; one box is `box` whole rows.  256-byte rows land
// as [8-row group][128-byte half][8 rows][128 B], 128-byte rows as they are.
template <int D, bool E4>
bool pool_map(CUtensorMap *map, const void *pool, int64_t rows, int box) {
    const auto type = E4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if constexpr (!E4 && D == 128) {
        const cuuint64_t dim[4] = {64, 8, 2, cuuint64_t(rows / 8)}, stride[3] = {256, 128, 2048};
        const cuuint32_t b[4] = {64, 8, 2, cuuint32_t(box / 8)};
        return encode(map, type, 4, pool, dim, stride, b);
    } else {
        const cuuint64_t dim[2] = {D, cuuint64_t(rows)}, stride[1] = {128};
        const cuuint32_t b[2] = {D, cuuint32_t(box)};
        return encode(map, type, 2, pool, dim, stride, b);
    }
}

Shape shape_of(int32_t hq, int32_t hkv) {
    const int group = hq / hkv;
    return {group, kRows / group};
}

struct Sizes {
    int64_t blocks, rows, slot_rows;
    int32_t ctas;
    size_t blocks_at, before, first, split, is_cut, cuts, piece0, pieces, o_part, lse_part, total;
};

// Most query blocks: every sequence's last one may be short.  Partial rows: two
// slots for each CTA, and two partials for every token of a block taken as a
// split item (its sequence's only or last block, at most tokens_per_tile of it).
Sizes sizes_of(const pkv_cache_desc &c, int64_t num_tokens, int32_t batch, int32_t hq) {
    const Shape sh = shape_of(hq, c.num_kv_heads);
    Sizes s;
    s.ctas = std::min(sm_count(), kMaxCtas);
    s.blocks = std::min(num_tokens, num_tokens / (2 * sh.tokens_per_tile) + batch);
    s.slot_rows = std::min<int64_t>(2 * kRows, 2 * num_tokens * sh.group);
    s.rows = 2 * s.ctas * s.slot_rows +
             2 * std::min(num_tokens, int64_t(batch) * sh.tokens_per_tile) * hq;
    const size_t items = size_t(s.blocks) * c.num_kv_heads;
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = (at + bytes + 255) & ~size_t(255);
        return here;
    };
    s.blocks_at = take(s.blocks * sizeof(Block));
    s.before = take((s.blocks + 1) * sizeof(int32_t));
    s.first = take((size_t(batch) + 1) * sizeof(int32_t));
    s.split = take(s.blocks * sizeof(int32_t));
    s.is_cut = take(items);
    s.cuts = take(s.ctas * sizeof(Cut));
    s.piece0 = take((s.ctas + 1) * sizeof(int32_t));
    // pieces: the rest's items (all of them when no round fits) and one more per cut
    s.pieces = take((items + s.ctas) * sizeof(Item));
    s.lse_part = take(s.rows * sizeof(float));
    s.o_part = take(size_t(s.rows) * c.head_dim_v * sizeof(float));
    s.total = at + 256;                  // the workspace may begin on any 16 bytes
    return s;
}

template <int D, bool E4, bool kWithhold>
int launch(const ChunkArgs &a, uint8_t *ws) {
    using C = Cfg<D, E4>;
    auto kernel = chunk_tc_kernel<D, E4, kWithhold>;
    const Shape sh = shape_of(a.num_q_heads, a.cache.num_kv_heads);
    const Sizes sz = sizes_of(a.cache, a.num_tokens, a.batch, a.num_q_heads);
    const Plan plan{reinterpret_cast<int32_t *>(ws),
                    reinterpret_cast<Block *>(ws + sz.blocks_at),
                    reinterpret_cast<int32_t *>(ws + sz.before),
                    reinterpret_cast<int32_t *>(ws + sz.first),
                    reinterpret_cast<int32_t *>(ws + sz.split),
                    ws + sz.is_cut,
                    reinterpret_cast<Cut *>(ws + sz.cuts),
                    reinterpret_cast<int32_t *>(ws + sz.piece0),
                    reinterpret_cast<Item *>(ws + sz.pieces),
                    reinterpret_cast<float *>(ws + sz.o_part),
                    reinterpret_cast<float *>(ws + sz.lse_part),
                    sz.ctas, int32_t(sz.slot_rows)};
    const int64_t rows = int64_t(a.cache.num_blocks) * a.cache.num_kv_heads * a.cache.block_size;
    const int box = std::min(a.cache.block_size, kKeys);
    CUtensorMap tq = {}, tk, tv;
    if (!pool_map<D, E4>(&tk, a.k_pool, rows, box) || !pool_map<D, E4>(&tv, a.v_pool, rows, box))
        return PKV_ERR_CUDA;
    if constexpr (!E4) {
        // boxes of one 128-byte column block of tokens_per_tile tokens' group heads
        const cuuint64_t dim[3] = {D, cuuint64_t(a.num_q_heads), cuuint64_t(a.num_tokens)};
        const cuuint64_t stride[2] = {D * 2, cuuint64_t(a.num_q_heads) * D * 2};
        const cuuint32_t b[3] = {64, cuuint32_t(sh.group), cuuint32_t(sh.tokens_per_tile)};
        if (!encode(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dim, stride, b))
            return PKV_ERR_CUDA;
    }
    static thread_local int configured_dev = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (configured_dev != dev) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(C::kSmem)) != cudaSuccess)
            return PKV_ERR_CUDA;
        configured_dev = dev;
    }
    int rc = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, a.stream, a, plan, sh);
    if (rc != PKV_OK) return rc;
    rc = launch_pdl(kernel, dim3(sz.ctas), dim3(C::kThreads), C::kSmem, a.stream, tq, tk, tv, a, plan,
                    sh);
    if (rc != PKV_OK) return rc;
    const int64_t merge_units = sz.blocks * a.cache.num_kv_heads * (kRows / kMergeRows) +
                                int64_t(sz.ctas) * (2 * kRows / kMergeRows);
    const int64_t merge_ctas = (merge_units + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
    return launch_pdl(chunk_merge_kernel<D>,
                      dim3(unsigned(std::min<int64_t>(merge_ctas, int64_t(sz.ctas) * 8))),
                      dim3(kMergeThreads), 0, a.stream, a, plan, sh);
}

template <bool kWithhold>
int launch_shape(const ChunkArgs &a, uint8_t *ws) {
    if (a.k_scale) return launch<128, true, kWithhold>(a, ws);
    return a.cache.head_dim_k == 128 ? launch<128, false, kWithhold>(a, ws)
                                     : launch<64, false, kWithhold>(a, ws);
}

}  // namespace

bool chunk_tc_supports(const pkv_cache_desc &c, int32_t num_q_heads, int32_t max_blocks, bool e4) {
    const int group = num_q_heads / c.num_kv_heads;
    const int least = e4 ? 16 : 8;
    const bool pow2 = c.block_size >= least && (c.block_size & (c.block_size - 1)) == 0;
    const int64_t rows = int64_t(c.num_blocks) * c.num_kv_heads * c.block_size;
    return c.head_dim_k == c.head_dim_v && (c.head_dim_k == 128 || (c.head_dim_k == 64 && !e4)) &&
           group <= kRows && pow2 && rows < (int64_t(1) << 31) - 1 &&
           int64_t(max_blocks) * c.block_size <= (int64_t(1) << 30);
}

size_t chunk_tc_workspace(const pkv_cache_desc &c, int64_t num_tokens, int32_t batch,
                          int32_t num_q_heads) {
    return sizes_of(c, num_tokens, batch, num_q_heads).total;
}

int launch_chunk_tc(const ChunkArgs &in, void *workspace) {
    ChunkArgs a = in;
    if (a.window == 0) a.sinks = 0;      // (both within the tables' capacity, below 2^30)
    uint8_t *ws = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(workspace) + 255) & ~uintptr_t(255));
    return a.withhold ? launch_shape<true>(a, ws) : launch_shape<false>(a, ws);
}

}  // namespace pkv
