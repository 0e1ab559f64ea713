// int4_ops.cu -- the 4-bit cache's append and block copies (its rows: pkv_int4.cuh).
//
// Append.  A row's scale needs the whole row before the first code, so a row stays in
// the registers of the lanes that loaded it: a lane holds units of 16 elements (two
// 16-byte vectors in, 8 bytes of codes out), a row's lanes find its extent by shuffles,
// and nothing is read twice.  A CTA takes one head's rows of neighbouring tokens, whose
// places in a block are neighbours too, so that codes and parameters are written in whole
// sectors.  Bound: memory, 2 D bytes in and D / 2 + 4 out a row, with about 7
// instructions an element close behind (logic instructions half of the time).  8 KV heads
// of 128: 64 tokens 1.9 us (latency), 8,191 tokens 10.9 us (0.58 of the copy rate: 1,024 CTAs,
// 760 at a time), 32,000 tokens 32.5 (0.77).  Six to eight CTAs an SM by fewer registers: 11.4
// to 12.7 us and 33.5 to 37.
//
// Block copies: memory, read and written once (8 KV heads of 128, blocks of 16 tokens: 16
// pairs 2.3 us, 1,000 12.7, 4,000 49.5, 0.42 of the copy rate).
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"
#include "pkv_int4.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    const uint16_t *k_new, *v_new;
    uint8_t *k_pool, *v_pool;
    uint32_t *k_params, *v_params;
    const int64_t *slots;
    uint32_t *status;
    int64_t num_tokens, num_slots;
    int32_t hkv, block_size, dk, dv;
    int32_t heads;                       // that a CTA takes in turn
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    f[0] = bf16_lo_to_f32(u.x); f[1] = bf16_hi_to_f32(u.x);
    f[2] = bf16_lo_to_f32(u.y); f[3] = bf16_hi_to_f32(u.y);
    f[4] = bf16_lo_to_f32(u.z); f[5] = bf16_hi_to_f32(u.z);
    f[6] = bf16_lo_to_f32(u.w); f[7] = bf16_hi_to_f32(u.w);
}

// LANES neighbouring lanes a row, UNITS units of 16 elements a lane: unit u of the row
// is the (u / LANES)-th of lane u mod LANES.  A lane's place in a row and its token's slot
// serve `heads` heads in turn, the next one's row on its way while one is stored.
template <int LANES, int UNITS>
__global__ void __launch_bounds__(kThreads) append_int4_kernel(const AppendArgs a) {
    constexpr int kRows = kThreads / LANES;              // tokens of a CTA's item
    const int c = threadIdx.x & (LANES - 1);
    pdl_wait();
    pdl_launch_dependents();
    const bool is_k = blockIdx.z == 0;
    const int d = is_k ? a.dk : a.dv;
    // grid.x: tokens, grid.y: heads, in strides; a whole warp goes through together (its
    // shuffles need all lanes)
    const int64_t tiles = (a.num_tokens + kRows - 1) / kRows;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t t = tile * kRows + threadIdx.x / LANES;
        const bool in = t < a.num_tokens;
        const int64_t slot = in ? a.slots[t] : -1;
        const uint16_t *token = (is_k ? a.k_new : a.v_new) + (in ? t : 0) * a.hkv * d + c * 16;
        for (int h0 = blockIdx.y * a.heads; h0 < a.hkv; h0 += gridDim.y * a.heads) {
            const int h1 = min(h0 + a.heads, a.hkv);
            uint4 raw[UNITS][2];
            auto load = [&](int h) {
#pragma unroll
                for (int u = 0; u < UNITS; ++u) {
                    raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
                    if (in && (c + u * LANES) * 16 < d) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(
                            token + int64_t(h) * d + u * LANES * 16);
                        raw[u][0] = src[0];
                        raw[u][1] = src[1];
                    }
                }
            };
            load(h0);
            const bool stored = slot >= 0 && slot < a.num_slots;
            if (slot >= a.num_slots && c == 0 && is_k && h0 == 0)
                raise_status(a.status, PKV_DEV_SLOT);
            // the row of head 0 (rows are numbered within 64 bits, blocks within 32)
            uint32_t block = 0;
            if (stored)
                block = a.num_slots <= UINT32_MAX ? uint32_t(slot) / uint32_t(a.block_size)
                                                  : uint32_t(slot / a.block_size);
            const int64_t row0 = int64_t(block) * a.hkv * a.block_size +
                                 (stored ? slot - int64_t(block) * a.block_size : 0);
            uint8_t *pool = (is_k ? a.k_pool : a.v_pool) + row0 * (d / 2) + c * 8;
            uint32_t *params = (is_k ? a.k_params : a.v_params) + row0;
            for (int h = h0; h < h1; ++h) {
                // two elements at a time
                uint32_t low2 = 0x7f807f80u, high2 = 0xff80ff80u;        // +inf, -inf
                uint4 now[UNITS][2];
#pragma unroll
                for (int u = 0; u < UNITS; ++u) {
                    const uint4 x = now[u][0] = raw[u][0], y = now[u][1] = raw[u][1];
                    if ((c + u * LANES) * 16 < d) {
                        low2 = min_nan_bf16x2(low2, min_nan_bf16x2(min_nan_bf16x2(x.x, x.y),
                                                                   min_nan_bf16x2(x.z, x.w)));
                        low2 = min_nan_bf16x2(low2, min_nan_bf16x2(min_nan_bf16x2(y.x, y.y),
                                                                   min_nan_bf16x2(y.z, y.w)));
                        high2 = max_nan_bf16x2(high2, max_nan_bf16x2(max_nan_bf16x2(x.x, x.y),
                                                                     max_nan_bf16x2(x.z, x.w)));
                        high2 = max_nan_bf16x2(high2, max_nan_bf16x2(max_nan_bf16x2(y.x, y.y),
                                                                     max_nan_bf16x2(y.z, y.w)));
                    }
                }
                if (h + 1 < h1) load(h + 1);
                const Int4Scale sc = int4_row_scale(
                    min_nan(bf16_lo_to_f32(low2), bf16_hi_to_f32(low2)),
                    max_nan(bf16_lo_to_f32(high2), bf16_hi_to_f32(high2)), LANES, 0xffffffffu);
                if (!stored) continue;
                const int64_t step = int64_t(h) * a.block_size;
#pragma unroll
                for (int u = 0; u < UNITS; ++u)
                    if ((c + u * LANES) * 16 < d) {
                        float x[8];
                        unpack8(now[u][0], x);
                        const uint32_t w0 = int4_codes8(x, sc);
                        unpack8(now[u][1], x);
                        *reinterpret_cast<uint2 *>(pool + step * (d / 2) + u * LANES * 8) =
                            make_uint2(w0, int4_codes8(x, sc));
                    }
                if (c == 0) params[step] = sc.params;
            }
        }
    }
}

// One CTA row (grid.x) a pair, grid.y shares its bytes.  Every CTA of a pair re-derives
// the same skip decision from the full pair list, so that no CTA writes a destination
// that another pair reads or writes.  16-byte vectors; the parameters in 4-byte words.
__global__ void copy_blocks_int4_kernel(uint4 *k_pool, uint32_t *k_params, uint4 *v_pool,
                                        uint32_t *v_params, const int32_t *src,
                                        const int32_t *dst, int32_t num_pairs,
                                        int32_t num_blocks, int64_t k_vecs, int64_t v_vecs,
                                        int64_t words, uint32_t *status) {
    pdl_wait();
    pdl_launch_dependents();
    const int32_t p = blockIdx.x;
    const int32_t s = src[p], d = dst[p];
    const bool in_range = s >= 0 && s < num_blocks && d >= 0 && d < num_blocks;
    int conflict = 0;
    for (int32_t q = threadIdx.x; q < num_pairs; q += blockDim.x)
        if (q != p && (dst[q] == d || src[q] == d)) conflict = 1;
    conflict = __syncthreads_or(conflict);
    if (!in_range || conflict) {
        if (blockIdx.y == 0 && threadIdx.x == 0)
            raise_status(status, in_range ? PKV_DEV_COPY_CONFLICT : PKV_DEV_BLOCK_ID);
        return;
    }
    if (s == d) return;
    const int64_t begin = blockIdx.y * int64_t(blockDim.x) + threadIdx.x;
    const int64_t step = int64_t(gridDim.y) * blockDim.x;
    for (int64_t u = begin; u < k_vecs + v_vecs; u += step) {
        if (u < k_vecs)
            k_pool[d * k_vecs + u] = k_pool[s * k_vecs + u];
        else
            v_pool[d * v_vecs + (u - k_vecs)] = v_pool[s * v_vecs + (u - k_vecs)];
    }
    for (int64_t u = begin; u < 2 * words; u += step) {
        if (u < words)
            k_params[d * words + u] = k_params[s * words + u];
        else
            v_params[d * words + (u - words)] = v_params[s * words + (u - words)];
    }
}

int valid_pools(const void *k_pool, const void *k_params, const void *v_pool,
                const void *v_params) {
    if (!k_pool || !k_params || !v_pool || !v_params) return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(k_params) || !aligned16(v_pool) || !aligned16(v_params))
        return PKV_ERR_ALIGNMENT;
    return PKV_OK;
}

}  // namespace

int validate_int4_cache(const pkv_cache_desc *c) {
    if (!c || c->num_blocks <= 0 || c->block_size < 1 || c->block_size > 256 ||
        c->num_kv_heads <= 0 || c->head_dim_k <= 0 || c->head_dim_v <= 0)
        return PKV_ERR_INVALID_ARG;
    if (c->head_dim_k % 32 || c->head_dim_v % 32 || c->head_dim_k > 1024 ||
        c->head_dim_v > 1024)
        return PKV_ERR_SHAPE;
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" int pkv_kv_append_int4(const pkv_cache_desc *cache, void *k_pool, void *k_params,
                                  void *v_pool, void *v_params, const void *k_new,
                                  const void *v_new, const int64_t *slot_mapping,
                                  int64_t num_tokens, pkv_stream_t stream) {
    int st = validate_int4_cache(cache);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    st = valid_pools(k_pool, k_params, v_pool, v_params);
    if (st == PKV_ERR_INVALID_ARG || !k_new || !v_new || !slot_mapping)
        return PKV_ERR_INVALID_ARG;
    if (st != PKV_OK || !aligned16(k_new) || !aligned16(v_new)) return PKV_ERR_ALIGNMENT;
    if (num_tokens > INT64_MAX / 4096 / cache->num_kv_heads) return PKV_ERR_SHAPE;
    AppendArgs a = {};
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    a.k_new = static_cast<const uint16_t *>(k_new);
    a.v_new = static_cast<const uint16_t *>(v_new);
    a.k_pool = static_cast<uint8_t *>(k_pool);
    a.v_pool = static_cast<uint8_t *>(v_pool);
    a.k_params = static_cast<uint32_t *>(k_params);
    a.v_params = static_cast<uint32_t *>(v_params);
    a.slots = slot_mapping;
    a.num_tokens = num_tokens;
    a.num_slots = int64_t(cache->num_blocks) * cache->block_size;
    a.hkv = cache->num_kv_heads;
    a.block_size = cache->block_size;
    a.dk = cache->head_dim_k;
    a.dv = cache->head_dim_v;
    // the fewest lanes that hold a row in one unit each, or 32 with two
    const int units = std::max(a.dk, a.dv) / 16;
    auto kernel = units <= 4    ? append_int4_kernel<4, 1>
                  : units <= 8  ? append_int4_kernel<8, 1>
                  : units <= 16 ? append_int4_kernel<16, 1>
                  : units <= 32 ? append_int4_kernel<32, 1>
                                : append_int4_kernel<32, 2>;
    const int lanes = units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32;
    const int rows = kThreads / lanes;
    const int64_t tiles = (num_tokens + rows - 1) / rows;
    // four heads a CTA where that leaves enough CTAs (8,191 tokens of 8 heads: 10.8 us, one
    // head a CTA 13.6)
    a.heads = tiles * 2 * a.hkv >= int64_t(sm_count()) * 16 ? std::min(4, a.hkv) : 1;
    const dim3 grid(unsigned(std::min<int64_t>(tiles, 1 << 20)),
                    unsigned(std::min((a.hkv + a.heads - 1) / a.heads, 65535)), 2);
    return launch_pdl(kernel, grid, dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), a);
}

extern "C" int pkv_copy_blocks_int4(const pkv_cache_desc *cache, void *k_pool, void *k_params,
                                    void *v_pool, void *v_params, const int32_t *src,
                                    const int32_t *dst, int32_t num_pairs,
                                    pkv_stream_t stream) {
    int st = validate_int4_cache(cache);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_INVALID_ARG;
    if (num_pairs == 0) return PKV_OK;
    st = valid_pools(k_pool, k_params, v_pool, v_params);
    if (st == PKV_ERR_INVALID_ARG || !src || !dst) return PKV_ERR_INVALID_ARG;
    if (st != PKV_OK) return st;
    if (num_pairs > 65535) return PKV_ERR_SHAPE;
    uint32_t *status = status_word();
    if (!status) return PKV_ERR_CUDA;
    const int64_t rows = int64_t(cache->num_kv_heads) * cache->block_size;
    const int64_t k_vecs = rows * cache->head_dim_k / 32, v_vecs = rows * cache->head_dim_v / 32;
    const int64_t per_pair = (k_vecs + v_vecs + kThreads - 1) / kThreads;
    const int64_t want =
        std::max<int64_t>(1, (int64_t(sm_count()) * 4 + num_pairs - 1) / num_pairs);
    const dim3 grid(num_pairs, unsigned(std::min<int64_t>({per_pair, want, 65535})));
    return launch_pdl(copy_blocks_int4_kernel, grid, dim3(kThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), static_cast<uint4 *>(k_pool),
                      static_cast<uint32_t *>(k_params), static_cast<uint4 *>(v_pool),
                      static_cast<uint32_t *>(v_params), src, dst, num_pairs, cache->num_blocks,
                      k_vecs, v_vecs, rows, status);
}
