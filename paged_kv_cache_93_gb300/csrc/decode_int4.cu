// decode_int4.cu -- decode attention over a 4-bit cache on tensor cores.
//
// Element d of token j's key is s_j c_jd + o_j (scale, offset, code), so
//     q . K_j = s_j (q . c_j) + o_j sum_d q_d,
//     sum_j p_j V_j = sum_j (p_j s'_j) c'_j + sum_j p_j o'_j
// and both products run over the codes themselves; scales and offsets are applied to the
// scores and to the weights, once a token.
//
// A row of 128 elements is 68 bytes, so an SM at full bandwidth meets 41 elements a clock
// and cannot afford an instruction for each.  Hence:
//  - A code needs no conversion.  Its bits 0..15 at bits 3-6 of an fp16 are the subnormal
//    code * 2^-21, and at bits 7-10 code * 2^-17 (up to 2047 an fp16's bits count evenly);
//    tensor cores take subnormals exactly.  A 32-bit word of 8 codes becomes four fp16
//    pairs with two shifts and four ANDs.  The factors 2^-21 and 16 go into the query and
//    into the result.  (At bits 0-3 and 4-7 it would be one shift.  But products are lined
//    up by their operands' exponents, and what a subnormal has in leading zeros is lost
//    below: scores off by 1e-5 instead of 1e-6.)
//  - Rows come by cp.async into a ring that belongs to one warp: 16-byte pieces may be
//    placed anywhere, no barrier couples the warps, and a warp's tiles are on their way
//    while it computes.
//  - Warp-level MMAs, which take the codes from registers as they come.  tcgen05 takes
//    operands from shared memory or tensor memory, where codes would be written first, as
//    fp16 in four times their bytes (120 of the 128 bytes a clock that shared memory moves,
//    with the reads).  As bytes they would be E4M3 numbers, code * 2^-9 exactly, in twice
//    their bytes, with query and weights as terms of E4M3; that form is not built, and at 8
//    and 16 rows, where the warps' products are the bound, it is what may be faster.
//  - Scores: A = 16 tokens x 16 elements, B = the query rows.  The order of the elements
//    within a product is free, so a lane takes D / 4 of a row in one load and the query
//    is laid out to match.
//  - Values: A = 16 elements x 16 tokens.  Again each lane takes whole words: lane group
//    g's word holds 8 elements, the n-th of which is row g of the n-th product.  Two
//    tokens' words interleave with two byte permutes into the pairs that the product
//    wants.
//  - A code is a positive number, and products' sums are cut off, not rounded, below
//    fp32's last place: thousands of tokens' values, which nearly cancel, would be lost
//    in a sum of codes that grows and grows (200,000 tokens: 1e-3 of the output).  So
//    half of the tokens enter the values' products as -p s' times 15 - code, which is an
//    exclusive-or in the instruction that masks the codes anyway, and 15 p s' goes to the
//    offsets' sum.  Which half: those whose place within 16 has an odd number of one
//    bits, a pattern that no regular spacing of tokens falls in with.
//  - Weights go from the scores' layout (token, row) to the values' (row, token) by
//    movmatrix.
// Query and weights are carried as two fp16 terms (22 bits): up to 4 rows as 8 columns
// (row, term), else two products.  A third term would be half as many products again; two
// leave errors of 2e-7 to 1.6e-6 of the result against 64 bits (45 shapes; the same in fp32
// throughout: 6e-8 to 3.3e-6), with ex2.approx (2^-22) for p.  One term would leave 2e-4
// to 6e-4.  The query is scaled by a power of two so that its
// largest element is 2^12..2^13; a row's weights p_j s'_j likewise, to 2^0..2^15, by a
// factor that follows their running maximum -- a key that weighs much may have values
// a millionth of the others'.
//
// Bound: the SM's instruction pipes, not memory.  A warp's tile of 32 tokens takes 32
// products at 4 rows, 64 at 8 and 128 at 16, 8 clocks of a quarter of the SM each (256,
// 512 and 1,024 clocks), in which fp32 instructions do not run and others run at about two
// thirds; about 250 logic instructions, 200 of them to take codes apart; and 130 fp32 ones.
// A quarter of an SM then takes 800, 1,000 and 1,700 clocks a tile, where memory would bring
// one in 730; the same batch read from L2 is as slow, and 8, 12 or 16 warps an SM make no
// difference.  What does not grow with the tokens -- launches, the chain length, table,
// rows, the end of the last CTAs and the merge -- is 9 us at 4 rows and 18 at 16.
//   16 of up to 128, 32 / 8 heads of 128        3.8 us (latency)
//   8 x 32K, 32 / 8                            55.6    (0.77 of the copy rate)
//   48 of up to 16K, 64 / 8                    96.1    (0.60)
//   8 x 32K, 4 tokens each, 32 / 8            117.9    (0.36; over an E4M3 cache 103.2)
//   1 x 200,000, 64 / 8                        58.5    (0.56)
//   32 x 4,095, 2 tokens each, 32 / 8 of 64    30.8    (0.37)
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_math.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3e38f;           // the running maximum of a row without a score
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;                 // tokens of a warp's step
constexpr int kResident = 3;              // CTAs of an SM
// Codes' places in a pair of fp16, and 1 / the value of a code of 1 in the first of them.
constexpr uint32_t kSmall = 0x00780078u, kLarge = 0x07800780u;
constexpr float kUp = 2097152.f;          // 2^21

// ROWS query rows of an item: 4 (as 8 columns of row and term), 8, or 16 (two tiles of 8).
template <int D, int ROWS>
struct Config {
    static constexpr int kRowBytes = D / 2;
    static constexpr int kWordsK = D / 32;            // words of a K row a lane takes
    static constexpr int kWordsV = D / 64;            // words of a V row a lane takes
    static constexpr int kProducts = 4 * kWordsV;     // products of 16 elements
    static constexpr bool kPacked = ROWS == 4;
    static constexpr int kCols = ROWS == 16 ? 2 : 1;  // tiles of 8 columns
    static constexpr int kTerms = kPacked ? 1 : 2;    // products a tile of columns
    static constexpr int kLaneRows = kPacked ? 1 : 2 * kCols;
    static constexpr int kCtas = kResident;
    static constexpr int kStages = D == 128 ? 3 : 4;  // (one more or less changes 2%)
    // The scores' sums of the two terms apart, where registers allow: fewer cut-offs on the
    // large one (16 rows of 128: none, as it takes 5% more time at 4 tokens a sequence).
    static constexpr int kChains = kPacked || (ROWS == 16 && D == 128) ? 1 : 2;
    // The query's fragments (the same for all the CTA's warps) in shared memory where the
    // registers hold more sums (8 rows of 128: 102 us against 105 for the ragged batch).
    static constexpr bool kSharedQuery = ROWS == 16 || (ROWS == 8 && D == 128);
    static_assert(!kSharedQuery || !kPacked, "a packed query is held by its lanes");
    // the query's fragments, each row's two factors, and what its scores' sums begin with
    static constexpr int kFragments = kWordsK * kCols * kTerms * 512;
    static constexpr int kQueryBytes = kFragments + ROWS * 12;
    static constexpr int kStageBytes = 2 * kTile * (kRowBytes + 4);
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kRings = kWarps * kWarpBytes;
    // the warps' outputs go over the rings at the end, a row's floats padded
    static constexpr int kOutRow = D + (kPacked ? 8 : 4);
    static constexpr int kMergeBytes = kWarps * ROWS * (kOutRow + 1) * 4;
    static constexpr int kSmem = (kRings > kMergeBytes ? kRings : kMergeBytes) + kQueryBytes;
    static_assert(kResident * (kSmem + 1024 + 256) <= 233472, "an SM's shared memory");
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}
// N words (1, 2 or 4) from an address aligned to them.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&x)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(a) : "memory");
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(x[0]), "=r"(x[1]) : "r"(a) : "memory");
    else
        x[0] = lds32(a);
}
__device__ __forceinline__ void sts_words(uint32_t a, const uint32_t (&x)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(a), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
}
__device__ __forceinline__ void sts_pair(uint32_t a, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void lds_pair(uint32_t a, float &x, float &y) {
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x), "=f"(y) : "r"(a) : "memory");
}
// D = A (16 x 16, row) * B (16 x 8, col) + D, fp16 inputs, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with nothing added.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Transposes the 8 x 8 matrix of 16-bit elements that the warp holds (lane 4 i + k: row
// i, columns 2 k and 2 k + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The place in its ring stage of a 16-byte piece of a tile's row, and the token (of
// eight) that is row m of a product.  Both are chosen so that the lanes of one pass of
// shared memory meet different banks: in the keys' reads rows of neighbouring m, whole;
// in the values' reads the rows of m = 0, 2, 4, 6 (or 1, 3, 5, 7), halves or whole.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    if constexpr (D == 128) return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
    else return row * 32 + (piece << 4);
}
template <int D>
__device__ __forceinline__ int token_at(int m) {
    if constexpr (D == 128) return m ^ ((m >> 1) & 1);         // 0 1 3 2 4 5 7 6
    else return (0x57463120 >> (4 * m)) & 7;                   // 0 2 1 3 6 4 7 5
}

// 2^n for n clamped to a normal number's range.
__device__ __forceinline__ float pow2(int n) {
    return __int_as_float((min(max(n, -126), 126) + 127) << 23);
}
// floor(log2 x) of a positive normal x
__device__ __forceinline__ int exponent(float x) {
    return ((__float_as_int(x) >> 23) & 255) - 127;
}

// Over the eight lanes that share lane mod 4.
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a CTA works on: the ROWS query rows from row0 on, of KV head `head` of sequence b (of
// length len), over the tokens begin .. end (begin a multiple of kTile); and where the
// result goes: chunk `part` of all rows, or (slot >= 0) the workspace's place `slot`.
struct Segment {
    int32_t b, head, row0, len, begin, end;
    int32_t part, slot;
};

// By the whole CTA.  `segment` says it again whenever it is called: what is wanted only
// before or after the loop holds no register in it.
template <int D, int ROWS, typename Say>
__device__ __forceinline__ void attend(const Int4DecodeArgs &a, uint8_t *smem, int block_shift,
                                       float *parts, float *part_lse, Say segment) {
    using C = Config<D, ROWS>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const pkv_cache_desc &c = a.cache;
    const int group = a.group, rows = group * a.q_tokens;
    const int head = segment().head, b = segment().b, row0 = segment().row0;
    const int begin = segment().begin, end = segment().end;
    // this warp's share, in whole tiles
    const int per = (end - begin + kWarps * kTile - 1) / (kWarps * kTile) * kTile;
    const int first = min(begin + warp * per, end), last = min(first + per, end);
    const int tiles = (last - first + kTile - 1) / kTile;

    // ---- the query, on its way: the CTA's threads take 8 neighbouring elements each
    constexpr int kEights = D / 8, kOctets = (ROWS * kEights + kThreads - 1) / kThreads;
    float4 octet[kOctets][2];
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        const int u = threadIdx.x + i * kThreads, r = row0 + u / kEights;
        octet[i][0] = octet[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u < ROWS * kEights && r < rows) {
            const int tok = r / group;
            const float4 *src = reinterpret_cast<const float4 *>(
                a.q + ((int64_t(b) * a.q_tokens + tok) * a.num_q_heads + head * group +
                       (r - tok * group)) * D + u % kEights * 8);
            octet[i][0] = src[0];
            octet[i][1] = src[1];
        }
    }

    // ---- the ring
    const uint32_t ring = smem_addr(smem) + warp * C::kWarpBytes;
    const int32_t *table = a.block_tables + int64_t(b) * a.max_blocks;
    const int last_block = last > first ? (last - 1) >> block_shift : -1;
    // The pool row where the i-th block's tokens of this head begin.  Past the last block,
    // and for a block id out of range, block 0's: its tokens are read and not used, or
    // the row is unspecified.
    auto entry = [&](int i) {
        uint32_t phys = 0;
        if (i <= last_block) {
            phys = uint32_t(table[i]);
            if (phys >= uint32_t(c.num_blocks)) {
                raise_status(a.status, PKV_DEV_BLOCK_ID);
                phys = 0;
            }
        }
        return (phys * uint32_t(c.num_kv_heads) + head) << block_shift;
    };
    // 32 table entries at a time, one a lane, and the next 32 on their way
    int window = first >> block_shift;
    uint32_t here = entry(window + lane), next = entry(window + 32 + lane);
    const int block_mask = (1 << block_shift) - 1;
    constexpr int kPieces = C::kRowBytes / 16;              // of a row
    constexpr int kPass = 32 / kPieces;                     // rows a pass of the warp
    const int my_row = lane / kPieces;
    const uint8_t *k_lane = a.k_pool + (lane % kPieces) * 16;
    const uint8_t *v_lane = a.v_pool + (lane % kPieces) * 16;
    const uint32_t my_piece = piece_at<D>(my_row, lane % kPieces);
    // parameters: four tokens a lane, K's by lanes 0-7, V's by lanes 8-15
    const int my_four = (lane & 7) * 4;
    const uint32_t *p_lane = lane < 8 ? a.k_params : a.v_params;
    uint32_t fill = ring;                                   // the stage that is filled next
    auto load = [&](int tile) {
        // (a tile begins at a multiple of its size, so its first row's block and place
        // and a row's own add up)
        const int j0 = first + tile * kTile;
        if ((j0 >> block_shift) - window >= 32) {
            window += 32;
            here = next;
            next = entry(window + 32 + lane);
        }
        const int block = (j0 >> block_shift) - window, inner = j0 & block_mask;
#pragma unroll
        for (int n = 0; n < kTile / kPass; ++n) {
            uint32_t at;
            if constexpr (kPass == 8)       // a block has 8 tokens at least: all one block
                at = __shfl_sync(0xffffffffu, here, block + (n * kPass >> block_shift)) +
                     (inner + (n * kPass & block_mask)) + my_row;
            else
                at = __shfl_sync(0xffffffffu, here, block + ((n * kPass + my_row) >> block_shift)) +
                     inner + ((n * kPass + my_row) & block_mask);
            const uint32_t to = fill + my_piece + n * kPass * C::kRowBytes;
            cp_async_16(to, k_lane + uint64_t(at) * C::kRowBytes);
            cp_async_16(to + kTile * C::kRowBytes, v_lane + uint64_t(at) * C::kRowBytes);
        }
        const uint32_t at = __shfl_sync(0xffffffffu, here, block + (my_four >> block_shift)) +
                            inner + (my_four & block_mask);
        if (lane < 16) cp_async_16(fill + 2 * kTile * C::kRowBytes + lane * 16, p_lane + at);
        fill += C::kStageBytes;
        if (fill == ring + C::kWarpBytes) fill = ring;
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
        if (i < tiles) load(i);
        cp_async_commit();
    }

    // ---- the query: B fragments of the tile's rows, scaled to 2^12 .. 2^13, in shared
    // memory and from there to every warp.  Word w of lane (g, t), elements
    // 8 (kWordsK t + w) + .. of its column's row: [2 step + half], step 0 takes 0, 4 and 1, 5;
    // step 1 takes 2, 6 and 3, 7; odd ones' codes come times 16.
    const uint32_t query = smem_addr(smem) + C::kSmem - C::kQueryBytes;
    uint32_t qf[C::kSharedQuery ? 1 : C::kCols][C::kTerms][C::kWordsK][4];
    const uint32_t shared_query = query + lane * 16;
    float factor[C::kLaneRows], offset_factor[C::kLaneRows];
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
        const int u = threadIdx.x + i * kThreads, r = u / kEights, piece = u % kEights;
        if (u >= ROWS * kEights) break;                    // (whole warps)
        const float x[8] = {octet[i][0].x, octet[i][0].y, octet[i][0].z, octet[i][0].w,
                            octet[i][1].x, octet[i][1].y, octet[i][1].z, octet[i][1].w};
        float sum = 0.f, amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum += x[e];
            amax = fmaxf(amax, fabsf(x[e]));
        }
#pragma unroll
        for (int o = 1; o < kEights; o <<= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        const int e = max(exponent(amax), -100);
        const float up = pow2(12 - e);
        uint32_t top[4], low[4];
#pragma unroll
        for (int e0 = 0; e0 < 4; ++e0) {
            const float s = e0 & 1 ? up * 0.0625f : up;
            const float y = x[e0] * s, z = x[e0 + 4] * s;
            top[e0] = pack_f16x2(y, z);
            low[e0] = pack_f16x2(y - f16_lo_to_f32(top[e0]), z - f16_hi_to_f32(top[e0]));
        }
        const int w = piece % C::kWordsK, column = C::kPacked ? 2 * r : r & 7;
        const uint32_t to = query + (w * C::kCols + (r >> 3)) * C::kTerms * 512 +
                            (4 * column + piece / C::kWordsK) * 16;
        sts_words(to, top);
        sts_words(to + (C::kPacked ? 64 : 512), low);
        // score = s (sum of products) * factor + o * offset_factor, in base-2 units; the
        // sum over the codes less 4, so that it passes through zero on its way: what products
        // cut off goes by the sum's size (errors 6% smaller over 45 shapes, in the larger ones
        // by up to a third, for 1% of the time)
        if (piece == 0) {
            sts_pair(query + C::kFragments + r * 8, a.scale * kLog2e * pow2(e - 12) * kUp,
                     a.scale * kLog2e * sum);
            sts32(query + C::kFragments + ROWS * 8 + r * 4, -4.f / kUp * up * sum);
        }
    }
    __syncthreads();
    // lane (g, t) has the scores of row t, or of rows 2 t, 2 t + 1
#pragma unroll
    for (int r = 0; r < C::kLaneRows; ++r) {
        const int row = C::kPacked ? t : 8 * (r >> 1) + 2 * t + (r & 1);
        lds_pair(query + C::kFragments + row * 8, factor[r], offset_factor[r]);
    }
    if constexpr (!C::kSharedQuery) {
#pragma unroll
        for (int n = 0; n < C::kCols; ++n)
#pragma unroll
            for (int term = 0; term < C::kTerms; ++term)
#pragma unroll
                for (int w = 0; w < C::kWordsK; ++w)
                    lds_words(shared_query + ((w * C::kCols + n) * C::kTerms + term) * 512,
                              qf[n][term][w]);
    }
    // every row sees the tokens before
    const int all_see = min(last, segment().len - a.q_tokens + 1);
    // tokens that the lane's r-th row sees
    auto sees = [&](int r) {
        const Segment seg = segment();
        const int row = seg.row0 + (C::kPacked ? t : 8 * (r >> 1) + 2 * t + (r & 1));
        return min(last, seg.len - a.q_tokens + 1 + min(row / group, a.q_tokens - 1));
    };

    // A row's running state, in base-2 units.  A token of score y has p = 2^(y - from);
    // l and off are the sums of p and of p o' (each lane its own tokens').  `from` is not
    // the largest score: it is moved so that the largest weight p s' lies between 1 and
    // 2^15, which the weights' fp16 terms need, a tile's sum of p o' within 2^24, and one of
    // p within 2^110.  It moves when one of them would leave that (`heaviest` and `top`: the
    // largest y + log2 max(s', |o'| / 32) and y that were met then), in the first tile and
    // seldom after it, so that the common tile needs no maximum over lanes.
    // Offsets count because rows of one value have scale 0, and then nothing but `top` held
    // p down: p o' had no bound.  At |o'| <= 32 s', as rows of many values have it, they
    // change nothing; beyond, weights below 2^10 lose nothing that p o' would not hide
    // (fp16's last place, 2^-25, against 2^15).  In 2^30 tokens off stays within 2^50; l,
    // which may get 2^110 a tile where all values are zero, is kept times 2^-16.
    // Values of unusual sizes put `from` far from the scores, which lose by it: 16 to 32
    // units off they are rounded by 2^-20 twice, 64 to 128 off (values of 2^-54 and less)
    // by 2^-18.  Scales and offsets times a power of two of the warp's own would mend that,
    // for 3% of everybody's time (8 x 32K 57.4 us); they are left as they are.
    float from[C::kLaneRows], l[C::kLaneRows], off[C::kLaneRows];
    float heaviest[C::kLaneRows], top[C::kLaneRows];
    float acc[C::kProducts][C::kCols][4];
#pragma unroll
    for (int r = 0; r < C::kLaneRows; ++r) {
        from[r] = heaviest[r] = top[r] = kNone;
        l[r] = off[r] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < C::kProducts; ++i)
#pragma unroll
        for (int n = 0; n < C::kCols; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[i][n][x] = 0.f;
    const int tok = token_at<D>(g);                // the lane's token of the first 8
    // complemented tokens (rows 0-7 of a product; rows 8-15 are the other way round): the
    // lane's own in the scores' layout, and those of its pair in the values'
    const int odd_row = __popc(g) & 1;
    const uint32_t flips = t == 0 || t == 3 ? kSmall & 0xffff0000u : kSmall & 0xffffu;
    const uint32_t my_k = D == 128 ? piece_at<D>(tok, t) : piece_at<D>(tok, 0) + 8 * t;
    auto word_at = [&](int row) {
        return kTile * C::kRowBytes +
               (D == 128 ? piece_at<D>(row, g >> 1) + (g & 1) * 8 : piece_at<D>(row, 0) + g * 4);
    };
    const uint32_t my_v0 = word_at(token_at<D>(2 * t)), my_v1 = word_at(token_at<D>(2 * t + 1));
    // the sums over the codes of a tile's keys: scores of tokens tok + 8 k
    float s[2][C::kCols][4], low[2][C::kCols][4];
    auto dot_keys = [&](uint32_t stage) {
        uint32_t kw[4][C::kWordsK];
#pragma unroll
        for (int k = 0; k < 4; ++k) lds_words(stage + my_k + 8 * k * C::kRowBytes, kw[k]);
        float start[C::kLaneRows];
#pragma unroll
        for (int r = 0; r < C::kLaneRows; ++r) {
            const int row = C::kPacked ? t : 8 * (r >> 1) + 2 * t + (r & 1);
            start[r] = __uint_as_float(lds32(query + C::kFragments + ROWS * 8 + row * 4));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < C::kCols; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    low[h][n][e] = 0.f;
                    if constexpr (C::kPacked) s[h][n][e] = e & 1 ? 0.f : start[0];
                    else s[h][n][e] = start[2 * n + (e & 1)];
                }
#pragma unroll
        for (int w = 0; w < C::kWordsK; ++w) {
            uint32_t q[C::kCols][C::kTerms][4];
#pragma unroll
            for (int n = 0; n < C::kCols; ++n)
#pragma unroll
                for (int term = 0; term < C::kTerms; ++term) {
                    if constexpr (C::kSharedQuery) {
                        lds_words(shared_query + ((w * C::kCols + n) * C::kTerms + term) * 512,
                                  q[n][term]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) q[n][term][e] = qf[n][term][w][e];
                    }
                }
#pragma unroll
            for (int step = 0; step < 2; ++step)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = step ? kw[2 * h][w] >> 5 : kw[2 * h][w] << 3;
                    const uint32_t v = step ? kw[2 * h + 1][w] >> 5 : kw[2 * h + 1][w] << 3;
                    const uint32_t a0 = u & kSmall, a2 = u & kLarge;
                    const uint32_t a1 = v & kSmall, a3 = v & kLarge;
#pragma unroll
                    for (int n = 0; n < C::kCols; ++n)
#pragma unroll
                        for (int term = 0; term < C::kTerms; ++term)
                            mma_f16(C::kChains == 2 && term ? low[h][n] : s[h][n], a0, a1, a2, a3,
                                    q[n][term][2 * step], q[n][term][2 * step + 1]);
                }
        }
        if constexpr (C::kChains == 2)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < C::kCols; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[h][n][e] += low[h][n][e];
    };
    uint32_t stage = ring;
    for (int i = 0; i < tiles; ++i) {
        cp_async_wait<C::kStages - 2>();
        __syncwarp();                  // the tile is there; the stage before it is free
        if (i + C::kStages - 1 < tiles) load(i + C::kStages - 1);
        cp_async_commit();
        dot_keys(stage);
        const uint32_t params = stage + 2 * kTile * C::kRowBytes + tok * 4;
        const int j0 = first + i * kTile;
        const bool tail = j0 + kTile > all_see;

        // ---- x[row][k]: the scores, less what is given
        float x[C::kLaneRows][4];
        uint32_t hidden = 0;           // bit 4 r + k
        auto scores = [&](const float (&less)[C::kLaneRows]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t kp = lds32(params + 32 * k);
                const float ks = bf16_lo_to_f32(kp), ko = fmaf(ks, 4.f, bf16_hi_to_f32(kp));
#pragma unroll
                for (int r = 0; r < C::kLaneRows; ++r) {
                    const float (&z)[4] = s[k >> 1][r >> 1];
                    const float dot = C::kPacked ? z[2 * (k & 1)] + z[2 * (k & 1) + 1]
                                                 : z[2 * (k & 1) + (r & 1)];
                    x[r][k] = fmaf(ks, dot * factor[r], fmaf(ko, offset_factor[r], -less[r]));
                }
            }
            // tokens past the end, or past what a row sees
            if (tail) {
#pragma unroll
                for (int r = 0; r < C::kLaneRows; ++r) {
                    const int n = sees(r);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (j0 + tok + 8 * k >= n) {
                            x[r][k] = -INFINITY;
                            hidden |= 1u << (4 * r + k);
                        }
                }
            }
        };
        // ---- the values' weights, over x, and the tile's sums of p and p o'
        float sum[C::kLaneRows], shift[C::kLaneRows];
        auto weigh = [&](auto in_tail) {
            bool leaves = false;       // a weight or a p is out of its range
#pragma unroll
            for (int r = 0; r < C::kLaneRows; ++r) sum[r] = shift[r] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t vp = lds32(params + (kTile + 8 * k) * 4);
                float vs = bf16_lo_to_f32(vp);
                const bool flipped = odd_row ^ (k & 1);
                const float vo = fmaf(vs, flipped ? 15.f : 0.f, bf16_hi_to_f32(vp));
                vs = flipped ? -vs : vs;
#pragma unroll
                for (int r = 0; r < C::kLaneRows; ++r) {
                    const float p = ex2_approx(x[r][k]);
                    sum[r] += p;
                    // (what is not seen may be anything)
                    if (decltype(in_tail)::value && (hidden >> (4 * r + k) & 1)) {
                        x[r][k] = 0.f;
                    } else {
                        x[r][k] = p * vs;
                        shift[r] = fmaf(p, vo, shift[r]);
                    }
                    leaves |= !(fabsf(x[r][k]) <= 32768.f);
                }
            }
#pragma unroll
            for (int r = 0; r < C::kLaneRows; ++r)
                leaves |= !(sum[r] <= 0x1p110f) || !(fabsf(shift[r]) <= 0x1p24f);
            return leaves;
        };
        bool move = i == 0;
        if (!move) {
            scores(from);
            const bool leaves = tail ? weigh(std::true_type{}) : weigh(std::false_type{});
            move = __any_sync(0xffffffffu, leaves);
        }
        if (move) {
            float by[C::kLaneRows];
#pragma unroll
            for (int r = 0; r < C::kLaneRows; ++r) by[r] = 0.f;
            scores(by);
#pragma unroll
            for (int r = 0; r < C::kLaneRows; ++r) {
                float y = kNone, w = kNone;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t vp = lds32(params + (kTile + 8 * k) * 4);
                    const float size = fmaxf(fabsf(bf16_lo_to_f32(vp)),
                                             fabsf(bf16_hi_to_f32(vp)) * 0.03125f);
                    y = fmaxf(y, x[r][k]);
                    if (!(hidden >> (4 * r + k) & 1) && size > 0.f)
                        w = fmaxf(w, x[r][k] + __log2f(size));
                }
                top[r] = fmaxf(top[r], group_max(y));
                heaviest[r] = fmaxf(heaviest[r], group_max(w));
                const float want = fmaxf(heaviest[r] - 10.f, top[r] - 100.f);
                const float now = fmaxf(from[r], fminf(want, top[r] + 100.f));
                by[r] = ex2_approx(from[r] - now);
                from[r] = now;
                l[r] *= by[r];
                off[r] *= by[r];
            }
#pragma unroll
            for (int p = 0; p < C::kProducts; ++p)
#pragma unroll
                for (int n = 0; n < C::kCols; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[p][n][e] *= by[C::kPacked ? 0 : 2 * n + (e & 1)];
            scores(from);
            if (tail) weigh(std::true_type{});
            else weigh(std::false_type{});
        }
#pragma unroll
        for (int r = 0; r < C::kLaneRows; ++r) {
            l[r] = fmaf(sum[r], 0x1p-16f, l[r]);
            off[r] += shift[r];
        }
        // ---- values: a tile's products by themselves, the small terms first, and added
        // with rounding to the running sums -- added there by the products they would lose
        // half a last place each time, always towards zero (1,000 products: 3e-5)
        uint32_t pb[2][C::kCols][C::kTerms][2];   // weights in the products' layout
        uint32_t both[2][C::kWordsV][2][2];       // [16 tokens][word][token pair][half]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (C::kPacked) {
                const float u = x[0][2 * h], v = x[0][2 * h + 1];
                const uint32_t hi = pack_f16x2(u, v);
                const uint32_t lo = pack_f16x2(u - f16_lo_to_f32(hi), v - f16_hi_to_f32(hi));
                pb[h][0][0][0] = transpose8(__byte_perm(hi, lo, 0x5410));
                pb[h][0][0][1] = transpose8(__byte_perm(hi, lo, 0x7632));
            } else {
#pragma unroll
                for (int n = 0; n < C::kCols; ++n)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float u = x[2 * n][2 * h + half], v = x[2 * n + 1][2 * h + half];
                        const uint32_t hi = pack_f16x2(u, v);
                        const uint32_t lo =
                            pack_f16x2(u - f16_lo_to_f32(hi), v - f16_hi_to_f32(hi));
                        pb[h][n][0][half] = transpose8(hi);
                        pb[h][n][C::kTerms - 1][half] = transpose8(lo);
                    }
            }
            // the four tokens of this lane, and their words
            uint32_t v0[C::kWordsV], v1[C::kWordsV], v2[C::kWordsV], v3[C::kWordsV];
            lds_words(stage + my_v0 + 16 * h * C::kRowBytes, v0);
            lds_words(stage + my_v1 + 16 * h * C::kRowBytes, v1);
            lds_words(stage + my_v0 + (16 * h + 8) * C::kRowBytes, v2);
            lds_words(stage + my_v1 + (16 * h + 8) * C::kRowBytes, v3);
#pragma unroll
            for (int w = 0; w < C::kWordsV; ++w) {
                both[h][w][0][0] = __byte_perm(v0[w], v1[w], 0x5410);
                both[h][w][0][1] = __byte_perm(v0[w], v1[w], 0x7632);
                both[h][w][1][0] = __byte_perm(v2[w], v3[w], 0x5410);
                both[h][w][1][1] = __byte_perm(v2[w], v3[w], 0x7632);
            }
        }
        // element n of word w for a pair of tokens: index 8 w + n
        auto element = [&](int h, int index, int pair) {
            const int n = index & 7;
            const uint32_t z = both[h][index >> 3][pair][n >> 2];
            const uint32_t flip = pair ? flips ^ kSmall : flips;
            const uint32_t y = (n & 2) ? z >> 5 : z << 3;
            return n & 1 ? (y & kLarge) ^ (flip << 4) : (y & kSmall) ^ flip;
        };
#pragma unroll
        for (int p = 0; p < C::kProducts; ++p) {
            uint32_t e[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                e[h][0] = element(h, p, 0);
                e[h][1] = element(h, p + C::kProducts, 0);
                e[h][2] = element(h, p, 1);
                e[h][3] = element(h, p + C::kProducts, 1);
            }
#pragma unroll
            for (int n = 0; n < C::kCols; ++n) {
                float z[4];
#pragma unroll
                for (int term = C::kTerms - 1; term >= 0; --term)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (term == C::kTerms - 1 && h == 0)
                            mma_f16_first(z, e[h][0], e[h][1], e[h][2], e[h][3], pb[h][n][term][0],
                                          pb[h][n][term][1]);
                        else
                            mma_f16(z, e[h][0], e[h][1], e[h][2], e[h][3], pb[h][n][term][0],
                                    pb[h][n][term][1]);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[p][n][i] += z[i];
            }
        }
        stage += C::kStageBytes;
        if (stage == ring + C::kWarpBytes) stage = ring;
    }

    // ---- the CTA's warps together: outputs, maxima and sums over the rings
    cp_async_wait<0>();
    __syncthreads();
    float *outs = reinterpret_cast<float *>(smem);            // [warp][ROWS][kOutRow]
    float *stats = outs + kWarps * ROWS * C::kOutRow;         // [warp][ROWS]
#pragma unroll
    for (int r = 0; r < C::kLaneRows; ++r) {
        // each warp's row by itself: its output, and log2 of its sum
        l[r] = group_sum(l[r]);
        off[r] = group_sum(off[r]);
        const bool some = l[r] > 0.f || l[r] != l[r];         // (a NaN score: a NaN row)
        // (l is the sum times 2^-16: so are off and the products)
        const float inv = some ? 1.f / l[r] : 0.f;
        off[r] *= 0x1p-16f;
        const int row = C::kPacked ? t : 8 * (r >> 1) + 2 * t + (r & 1);
        // the whole sum's logarithm; past what fp32 holds in two parts
        if (g == 0)
            stats[warp * ROWS + row] = !some               ? kNone
                                       : l[r] <= 0x1p100f ? from[r] + log2f(l[r] * 65536.f)
                                                          : from[r] + (log2f(l[r]) + 16.f);
        // The lane's neighbouring elements of the row, four at a time.  Eight lanes store at
        // once, two of g and four of t: the rows' padding and the odd g's order of fours
        // put them in banks of their own (one at a time they would meet 16 to a bank).
        float4 *o = reinterpret_cast<float4 *>(outs + (warp * ROWS + row) * C::kOutRow) +
                    2 * C::kWordsV * g;
        float y[2 * C::kProducts];
#pragma unroll
        for (int i = 0; i < 2 * C::kProducts; ++i) {
            const int p = i % C::kProducts, half = i / C::kProducts;
            const float z = C::kPacked ? acc[p][0][2 * half] + acc[p][0][2 * half + 1]
                                       : acc[p][r >> 1][2 * half + (r & 1)];
            y[i] = fmaf(z, i & 1 ? kUp * 0x1p-20f : kUp * 0x1p-16f, off[r]) * inv;
        }
#pragma unroll
        for (int c = 0; c < C::kProducts / 2; c += 2) {
            const float4 u = make_float4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
            const float4 v = make_float4(y[4 * c + 4], y[4 * c + 5], y[4 * c + 6], y[4 * c + 7]);
            o[c + (g & 1)] = g & 1 ? v : u;
            o[c + 1 - (g & 1)] = g & 1 ? u : v;
        }
    }
    __syncthreads();
    const Segment seg = segment();
    float *out = seg.slot < 0 ? a.out_part : parts + int64_t(seg.slot) * ROWS * D;
    float *lse = seg.slot < 0 ? a.lse_part : part_lse + int64_t(seg.slot) * ROWS;
    for (int u = threadIdx.x; u < ROWS * (D / 4); u += kThreads) {
        const int r = u / (D / 4), e = (u - r * (D / 4)) * 4;
        if (seg.row0 + r >= rows) break;
        float most = kNone, all = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, stats[w * ROWS + r]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float z = stats[w * ROWS + r];
            const float by = z == kNone ? 0.f : ex2_approx(z - most);
            const float4 y =
                *reinterpret_cast<const float4 *>(outs + (w * ROWS + r) * C::kOutRow + e);
            all += by;
            o.x = fmaf(by, y.x, o.x); o.y = fmaf(by, y.y, o.y);
            o.z = fmaf(by, y.z, o.z); o.w = fmaf(by, y.w, o.w);
        }
        const bool some = all != 0.f;
        const float inv = some ? 1.f / all : 0.f;
        int64_t to = r;
        if (seg.slot < 0) {
            const int token = (seg.row0 + r) / group;
            to = ((int64_t(seg.part) * a.batch + seg.b) * a.q_tokens + token) * a.num_q_heads +
                 seg.head * group + (seg.row0 + r - token * group);
        }
        *reinterpret_cast<float4 *>(out + to * D + e) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (e == 0)
            lse[to] = seg.slot >= 0 ? (some ? most + log2f(all) : kNone)
                      : some        ? (most + log2f(all)) * kLn2
                                    : -INFINITY;
    }
}

// The sequence's length; one that is not valid counts as 0.  (L2: for reads before the
// wait for the kernel before, which alone makes an older line of the first cache go.)
template <bool L2 = false>
__device__ __forceinline__ int length_of(const Int4DecodeArgs &a, int block_shift, int b) {
    const int32_t len = L2 ? __ldcg(a.seq_lens + b) : a.seq_lens[b];
    return len < 0 || len > (int64_t(a.max_blocks) << block_shift) ? 0 : len;
}
__device__ __forceinline__ void check_length(const Int4DecodeArgs &a, int block_shift, int b) {
    const int32_t len = a.seq_lens[b];
    if (len < a.flag_below || len < 0 || len > (int64_t(a.max_blocks) << block_shift))
        raise_status(a.status, PKV_DEV_SEQ_LEN);
}

// Lengths and tables into L2, a line a thread, while the kernel before this one ends: the
// first tile waits for a length, then for a table entry, then for its rows.
__device__ __forceinline__ void prefetch_tables(const Int4DecodeArgs &a) {
    const int64_t at = (blockIdx.x * int64_t(kThreads) + threadIdx.x) * 128;
    const int64_t lens = int64_t(a.batch) * 4, tables = lens * a.max_blocks;
    if (at < lens)
        asm volatile("prefetch.global.L2 [%0];"
                     ::"l"(reinterpret_cast<const char *>(a.seq_lens) + at));
    if (at < tables)
        asm volatile("prefetch.global.L2 [%0];"
                     ::"l"(reinterpret_cast<const char *>(a.block_tables) + at));
}

// ---- a given number of splits: one CTA for each (sequence, KV head, split, tile of rows),
// the last fastest, so that CTAs that read the same tokens run together
template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, Config<D, ROWS>::kCtas)
decode_int4_kernel(const Int4DecodeArgs a, int row_tiles, int block_shift) {
    extern __shared__ __align__(128) uint8_t smem[];
    prefetch_tables(a);
    pdl_wait();
    pdl_launch_dependents();
    uint32_t item = blockIdx.x;
    const int row0 = int(item % row_tiles) * ROWS;
    item /= row_tiles;
    const int split = int(item % a.num_splits);
    item /= a.num_splits;
    const int head = int(item % a.cache.num_kv_heads), b = int(item / a.cache.num_kv_heads);
    if (threadIdx.x == 0 && split == 0 && row0 == 0 && head == 0) check_length(a, block_shift, b);
    const int64_t len = length_of(a, block_shift, b);
    const int64_t chunk = 64 * ((len + 64LL * a.num_splits - 1) / (64LL * a.num_splits));
    const int begin = int(min(split * chunk, len)), end = int(min((split + 1) * chunk, len));
    const Segment seg{b, head, row0, int(len), begin, end, split, -1};
    attend<D, ROWS>(a, smem, block_shift, nullptr, nullptr, [&]() { return seg; });
}

// ---- the library's own plan: the CTAs that the device holds at once share the batch's
// work evenly, whatever the lengths.
//
// A unit is a (sequence, KV head, tile of rows): n = ceil(length / 128) steps of a CTA's
// four warps, and kStart more for the start and end of one more piece of work.  The units
// lie one after another on a line of T = sum (n + kStart); CTA i of C takes
// [floor(i T / C), floor((i + 1) T / C)) of it, so it meets the end of one unit, perhaps
// some whole ones, and the beginning of another.  A whole unit goes straight to the
// output; the parts of others go to the workspace (CTA i's at 2 i, or 2 i + 1 if it is the
// unit's first) and are merged by the next kernel, which finds them from the lengths by
// itself.  Where all sequences have the same number of steps, C is a multiple of the units
// if one is near enough, so that no CTA meets two (8 x 32K, 64 units: 448 of 456 CTAs).
constexpr int kStep = kWarps * kTile;
// (1, 2, 3, 4: 48 of up to 16K 105, 97, 97, 98 us; 128 of up to 8K 120, 117, 104, 105)
constexpr int kStart = 3;
constexpr int kMaxPlanned = 512;           // sequences
constexpr int kManyUnits = 3;              // a CTA

__device__ __forceinline__ int steps_of(int len) {
    return int((uint32_t(len) + kStep - 1) / kStep);
}

// The line, as the lanes of a warp see it: each has the sequences b0 .. b1, the first of
// which begins at `start`.
struct Line {
    int64_t total, start, end;
    int32_t ctas;                          // that have a share of it
    int32_t extra;                         // what a unit has on the line beside its steps
    int32_t b0, b1;
};

template <bool L2 = false>
__device__ __forceinline__ Line line_of(const Int4DecodeArgs &a, int block_shift, int heads,
                                        int ctas, int even) {
    const int lane = threadIdx.x & 31, per = (a.batch + 31) / 32;
    Line line;
    line.b0 = min(lane * per, a.batch);
    line.b1 = min(line.b0 + per, a.batch);
    int64_t mine = 0;
    int least = INT32_MAX, most = 0;
#pragma unroll 8
    for (int b = line.b0; b < line.b1; ++b) {
        const int n = steps_of(length_of<L2>(a, block_shift, b));
        least = min(least, n);
        most = max(most, n);
        mine += n + kStart;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
    // (a share that begins with a unit has no more to start than any other; `even` is the
    // largest multiple of the units within `ctas`)
    line.extra = least == most && least > 0 && 10 * even >= 9 * ctas ? 0 : kStart;
    if (line.extra == 0) {
        mine -= int64_t(kStart) * (line.b1 - line.b0);
        upto -= int64_t(kStart) * line.b1;
    }
    line.total = (all - (line.extra ? 0 : int64_t(kStart) * a.batch)) * heads;
    // each CTA has a place of the line or more
    line.ctas = int(min(int64_t(line.extra ? ctas : even), line.total));
    line.start = (upto - mine) * heads;
    line.end = upto * heads;
    return line;
}

// The CTA whose share has a place of the line: the largest i with i total / ctas < place + 1.
__device__ __forceinline__ int cta_of(int64_t place, int64_t total, int ctas) {
    return int(((place + 1) * ctas - 1) / total);
}

struct Share {                             // a CTA's share of the line, and where it stands
    int64_t at, to, start;                 // start: of sequence b
    int32_t b, len, extra;
};

// The next part of a unit with something to do (b < 0: none).
__device__ __forceinline__ Segment next_segment(const Int4DecodeArgs &a, int block_shift,
                                                int row_tiles, int rows, Share &share) {
    const int heads = a.cache.num_kv_heads * row_tiles;     // units of a sequence
    Segment seg = {};
    seg.b = -1;
    while (share.at < share.to) {
        const int n = steps_of(share.len), cost = n + share.extra;
        const int64_t in = share.at - share.start;
        if (in >= int64_t(cost) * heads) {
            share.start += int64_t(cost) * heads;
            share.len = length_of(a, block_shift, ++share.b);
            continue;
        }
        const int unit = in <= INT32_MAX ? int(in) / cost : int(in / cost);
        const int64_t unit_at = share.start + int64_t(unit) * cost;
        const int64_t stop = min(share.to, unit_at + cost);
        const int s0 = max(0, int(share.at - unit_at) - share.extra);
        const int s1 = max(0, int(stop - unit_at) - share.extra);
        const bool empty = n == 0 && share.at == unit_at;
        share.at = stop;
        // (a sequence without tokens: whoever has its first place writes its rows)
        if (s1 > s0 || empty) {
            seg.b = share.b;
            seg.head = unit / row_tiles;
            seg.row0 = (unit - seg.head * row_tiles) * rows;
            seg.len = share.len;
            seg.begin = s0 * kStep;
            seg.end = int(min(int64_t(s1) * kStep, int64_t(share.len)));
            seg.slot = s0 == 0 && s1 == n ? -1 : 2 * int(blockIdx.x) + (s0 == 0 ? 1 : 0);
            break;
        }
    }
    return seg;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads, Config<D, ROWS>::kCtas)
decode_int4_planned_kernel(const Int4DecodeArgs a, int row_tiles, int block_shift, int even,
                           float *parts, float *part_lse) {
    extern __shared__ __align__(128) uint8_t smem[];
    // (in shared memory, as the registers belong to the work itself)
    __shared__ Share s_share;
    __shared__ Segment s_seg;
    prefetch_tables(a);
    pdl_wait();
    pdl_launch_dependents();
    {
        // Each warp by itself, without a barrier: the sequence in which this CTA's share
        // begins.
        const int lane = threadIdx.x & 31, heads = a.cache.num_kv_heads * row_tiles;
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b < a.batch; b += kThreads) check_length(a, block_shift, b);
        const Line line = line_of(a, block_shift, heads, int(gridDim.x), even);
        if (blockIdx.x >= line.ctas) return;
        Share share;
        share.extra = line.extra;
        // floor(i total / ctas) = i q + floor(i r / ctas), and the next (ctas^2 is far below
        // 2^31)
        const int cta = int(blockIdx.x), ctas = line.ctas;
        const int64_t q = line.total <= INT32_MAX ? int(line.total) / ctas : line.total / ctas;
        const int r = int(line.total - q * ctas), more = cta * r / ctas;
        share.at = cta * q + more;
        share.to = share.at + q + (cta * r - more * ctas + r >= ctas ? 1 : 0);
        // the lane whose sequences it begins in
        share.start = line.start;
        share.b = line.b0;
        share.len = 0;
        const bool here = line.start <= share.at && share.at < line.end;
        if (here)
            for (;; ++share.b) {
                share.len = length_of(a, block_shift, share.b);
                const int64_t cost = int64_t(steps_of(share.len) + share.extra) * heads;
                if (share.at < share.start + cost) break;
                share.start += cost;
            }
        const int owner = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        share.start = __shfl_sync(0xffffffffu, share.start, owner);
        share.b = __shfl_sync(0xffffffffu, share.b, owner);
        share.len = __shfl_sync(0xffffffffu, share.len, owner);
        if (threadIdx.x < 32) {
            const Segment seg = next_segment(a, block_shift, row_tiles, ROWS, share);
            if (lane == 0) {
                s_seg = seg;
                s_share = share;
            }
        }
    }
    __syncthreads();
    while (s_seg.b >= 0) {
        attend<D, ROWS>(a, smem, block_shift, parts, part_lse,
                        [&]() { return s_seg; });
        __syncthreads();           // nobody wants the segment any more, and the rings are free
        if (threadIdx.x == 0) {
            Share share = s_share;
            s_seg = next_segment(a, block_shift, row_tiles, ROWS, share);
            s_share = share;
        }
        __syncthreads();
    }
}

// Merges the units in parts.  A CTA has a unit's rows RB at a time, each by kThreads / RB
// threads: D / 4 threads with four elements of the row each, times the groups that take
// its parts in turn.  Many parts (one row a CTA) want groups, few parts rows.
template <int D, int ROWS, int RB>
__global__ void __launch_bounds__(kThreads)
int4_merge_kernel(const Int4DecodeArgs a, int row_tiles, int block_shift, int grid, int even,
                  const float *parts, const float *part_lse) {
    constexpr int kLanes = D / 4, kGroups = kThreads / RB / kLanes;
    __shared__ float4 s_out[RB][kGroups][kLanes];
    __shared__ float s_top[RB][kGroups], s_sum[RB][kGroups];
    // Which CTAs have the unit's steps.  This goes before the wait: the kernel before this
    // one lets it begin only after waiting for what came earlier, and does not write lengths.
    const int heads = a.cache.num_kv_heads * row_tiles;
    const int b = int(blockIdx.x) / heads, unit = int(blockIdx.x) - b * heads;
    __shared__ int s_first, s_parts;
    if (threadIdx.x < 32) {
        const Line line = line_of<true>(a, block_shift, heads, grid, even);
        int64_t at = line.start;
        int steps = 0;
        if (line.b0 <= b && b < line.b1) {
#pragma unroll 8
            for (int i = line.b0; i < b; ++i)
                at += int64_t(steps_of(length_of<true>(a, block_shift, i)) + line.extra) * heads;
            steps = steps_of(length_of<true>(a, block_shift, b));
            at += int64_t(unit) * (steps + line.extra) + line.extra;      // of its first step
            int first = 0, parts = 0;
            if (steps) {
                first = cta_of(at, line.total, line.ctas);
                parts = cta_of(at + steps - 1, line.total, line.ctas) - first + 1;
            }
            s_first = first;
            s_parts = parts;
        }
    }
    const int rb = threadIdx.x / (kThreads / RB), e = threadIdx.x % kLanes;
    const int grp = threadIdx.x % (kThreads / RB) / kLanes;
    const int r = blockIdx.y * RB + rb;                       // of the unit's tile
    const int group = a.group, head = unit / row_tiles;
    const int row = (unit - head * row_tiles) * ROWS + r, token = row / group;
    const int64_t to = (int64_t(b) * a.q_tokens + token) * a.num_q_heads + head * group +
                       (row - token * group);
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int first = s_first, num_parts = s_parts;
    if (num_parts < 2) return;                                // (written by the one CTA)
    float top = kNone, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 10;
    for (int p0 = grp; p0 < num_parts; p0 += kGroups * kAhead) {
        float z[kAhead];
        float4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            // (past the last part: that one again, without weight -- loads that hang on no
            // condition go out together)
            const int p = min(p0 + u * kGroups, num_parts - 1);
            const int slot = 2 * (first + p) + (p == 0 ? 1 : 0);
            z[u] = part_lse[slot * ROWS + r];
            x[u] = reinterpret_cast<const float4 *>(parts)[(slot * ROWS + r) * kLanes + e];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (p0 + u * kGroups >= num_parts) z[u] = kNone;
        float now = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) now = fmaxf(now, z[u]);
        const float by = ex2_approx(top - now);
        sum *= by;
        o = make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float w = z[u] == kNone ? 0.f : ex2_approx(z[u] - now);
            sum += w;
            o.x = fmaf(w, x[u].x, o.x); o.y = fmaf(w, x[u].y, o.y);
            o.z = fmaf(w, x[u].z, o.z); o.w = fmaf(w, x[u].w, o.w);
        }
        top = now;
    }
    if constexpr (kGroups > 1) {
        s_out[rb][grp][e] = o;
        if (e == 0) {
            s_top[rb][grp] = top;
            s_sum[rb][grp] = sum;
        }
        __syncthreads();
        if (grp != 0) return;
        float most = kNone, all = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) most = fmaxf(most, s_top[rb][i]);
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const float w = ex2_approx(s_top[rb][i] - most);
            const float4 x = s_out[rb][i][e];
            all = fmaf(w, s_sum[rb][i], all);
            o.x = fmaf(w, x.x, o.x); o.y = fmaf(w, x.y, o.y);
            o.z = fmaf(w, x.z, o.z); o.w = fmaf(w, x.w, o.w);
        }
        top = most;
        sum = all;
    }
    if (token >= a.q_tokens) return;
    const bool some = sum != 0.f;
    const float inv = some ? 1.f / sum : 0.f;
    *reinterpret_cast<float4 *>(a.out_part + to * D + 4 * e) =
        make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (e == 0) a.lse_part[to] = some ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

// Rows of an item for `rows` in all.
int tile_rows(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

int shift_of(int block_size) {
    int shift = 0;
    while ((1 << shift) < block_size) ++shift;
    return shift;
}

int row_tiles(const pkv_cache_desc &c, int32_t num_q_heads, int32_t q_tokens) {
    const int rows = num_q_heads / c.num_kv_heads * q_tokens;
    return (rows + tile_rows(rows) - 1) / tile_rows(rows);
}

template <int D, int ROWS>
int launch(const Int4DecodeArgs &a, void *workspace) {
    using C = Config<D, ROWS>;
    static_assert(C::kCtas == kResident, "the plan's CTAs are those that run at once");
    const int tiles = row_tiles(a.cache, a.num_q_heads, a.q_tokens);
    const int shift = shift_of(a.cache.block_size);
    // once a device and thread: room for the rings
    static thread_local int configured = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && configured != dev) {
        e = cudaFuncSetAttribute(decode_int4_kernel<D, ROWS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(decode_int4_planned_kernel<D, ROWS>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e == cudaSuccess) configured = dev;
    }
    if (e != cudaSuccess) return cuda_status(e);
    if (a.num_splits > 0) {
        const int64_t items = int64_t(a.batch) * a.cache.num_kv_heads * tiles * a.num_splits;
        return launch_pdl(decode_int4_kernel<D, ROWS>, dim3(unsigned(items)), dim3(kThreads),
                          C::kSmem, a.stream, a, tiles, shift);
    }
    const int ctas = sm_count() * kResident, units = a.batch * a.cache.num_kv_heads * tiles;
    const int even = ctas / units * units;
    float *parts = static_cast<float *>(workspace);
    float *part_lse = parts + size_t(2) * ctas * ROWS * D;
    const int st = launch_pdl(decode_int4_planned_kernel<D, ROWS>, dim3(ctas), dim3(kThreads),
                              C::kSmem, a.stream, a, tiles, shift, even, parts, part_lse);
    if (st != PKV_OK) return st;
    // more than about nine parts a unit: a row a CTA, its parts in groups
    constexpr int kRows = std::min(ROWS, 512 / D);
    const bool many = ctas > 8 * units;
    return launch_pdl(many ? int4_merge_kernel<D, ROWS, 1> : int4_merge_kernel<D, ROWS, kRows>,
                      dim3(units, many ? ROWS : ROWS / kRows), dim3(kThreads), 0,
                      a.stream, a, tiles, shift, ctas, even, static_cast<const float *>(parts),
                      static_cast<const float *>(part_lse));
}

}  // namespace

bool int4_kernel_supports(const pkv_cache_desc &c, int32_t batch, int32_t num_q_heads,
                          int32_t q_tokens, int32_t max_blocks) {
    const int32_t bs = c.block_size;
    if (c.head_dim_k != c.head_dim_v || (c.head_dim_k != 64 && c.head_dim_k != 128) || bs < 8 ||
        (bs & (bs - 1)) != 0)
        return false;
    // pool rows are numbered within 32 bits, a sequence's tokens within 30, items within 31
    // at any split count
    if (int64_t(c.num_blocks) * c.num_kv_heads * bs > int64_t(UINT32_MAX)) return false;
    if (int64_t(max_blocks) * bs > (1 << 30)) return false;
    const int64_t rows = int64_t(num_q_heads) / c.num_kv_heads * q_tokens;
    return int64_t(batch) * c.num_kv_heads * ((rows + 3) / 4) * 256 <= INT32_MAX;
}

size_t int4_plan_workspace(const pkv_cache_desc &c, int32_t batch, int32_t num_q_heads,
                           int32_t q_tokens, int32_t max_blocks) {
    if (batch > kMaxPlanned) return 0;
    const int64_t ctas = int64_t(sm_count()) * kResident;
    const int64_t units = int64_t(batch) * c.num_kv_heads * row_tiles(c, num_q_heads, q_tokens);
    // Where a plan costs more than it evens out, a CTA a unit: sequences of a few steps at
    // most (16 of up to 128 tokens: 3.8 us, planned 7.1; the host knows the tables' width and
    // not the lengths, so short sequences in wide tables are planned); many units, which even
    // out by themselves (1,024 of up to 8K tokens 126 us, planned 103; 1,280 of up to 2K 48.7
    // and 50.9; 2,048 of up to 2K 69.4 and 82); many sequences, which every CTA adds up (512
    // of up to 8K and one KV head 107 us, planned 89; 1,024 of them 172 and 198).
    const int64_t tokens = int64_t(max_blocks) * c.block_size;
    if (tokens <= 4 * kStep || units > kManyUnits * ctas) return 0;
    const int rows = tile_rows(num_q_heads / c.num_kv_heads * q_tokens);
    return size_t(ctas) * 2 * rows * (c.head_dim_v + 1) * sizeof(float);
}

int launch_decode_int4(const Int4DecodeArgs &a, void *workspace) {
    const int rows = tile_rows(a.num_q_heads / a.cache.num_kv_heads * a.q_tokens);
    if (a.cache.head_dim_k == 128)
        return rows == 4   ? launch<128, 4>(a, workspace)
               : rows == 8 ? launch<128, 8>(a, workspace)
                           : launch<128, 16>(a, workspace);
    return rows == 4   ? launch<64, 4>(a, workspace)
           : rows == 8 ? launch<64, 8>(a, workspace)
                       : launch<64, 16>(a, workspace);
}

}  // namespace pkv
