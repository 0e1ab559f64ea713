// int4_ops.cu -- the 4-bit cache's append and block copies (its rows: pkv_int4.cuh).
//
// Append.  A row's scale needs the whole row before the first code, so a row stays in
// the registers of the lanes that loaded it: a lane holds units of 16 elements (two
// 16-byte vectors in, 8 bytes of codes out), a row's lanes find its extent by shuffles,
// and nothing is read twice.  Bound: memory, 2 D bytes in and D / 2 + 4 out a row.
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
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    f[0] = bf16_lo_to_f32(u.x); f[1] = bf16_hi_to_f32(u.x);
    f[2] = bf16_lo_to_f32(u.y); f[3] = bf16_hi_to_f32(u.y);
    f[4] = bf16_lo_to_f32(u.z); f[5] = bf16_hi_to_f32(u.z);
    f[6] = bf16_lo_to_f32(u.w); f[7] = bf16_hi_to_f32(u.w);
}

// LANES neighbouring lanes a row, UNITS units of 16 elements a lane: unit u of the row
// is the (u / LANES)-th of lane u mod LANES.
template <int LANES, int UNITS>
__global__ void __launch_bounds__(kThreads) append_int4_kernel(const AppendArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kRows = kThreads / LANES;
    const int c = threadIdx.x & (LANES - 1);
    const int64_t rows = a.num_tokens * a.hkv;
    // K rows first, then V rows; a whole warp leaves together (its shuffles need all)
    const int64_t all = 2 * rows, steps = (all + kRows - 1) / kRows;
    for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
        int64_t r = step * kRows + threadIdx.x / LANES;
        const bool is_k = r < rows;
        const bool in = r < all;
        if (!is_k) r -= rows;
        const int d = is_k ? a.dk : a.dv;
        int64_t t = 0, slot = -1;
        if (in) {
            t = r / a.hkv;
            slot = a.slots[t];
            if (slot >= a.num_slots) {
                if (c == 0 && is_k && r == t * a.hkv) raise_status(a.status, PKV_DEV_SLOT);
                slot = -1;
            }
        }
        uint4 raw[UNITS][2];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int e = (c + u * LANES) * 16;
            if (slot >= 0 && e < d) {
                const uint4 *src =
                    reinterpret_cast<const uint4 *>((is_k ? a.k_new : a.v_new) + r * d + e);
                raw[u][0] = src[0];
                raw[u][1] = src[1];
            }
        }
        float low = INFINITY, high = -INFINITY, odd = 0.f;
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
            if (slot >= 0 && (c + u * LANES) * 16 < d) {
                float x[8];
                unpack8(raw[u][0], x);
                int4_extent8(x, low, high, odd);
                unpack8(raw[u][1], x);
                int4_extent8(x, low, high, odd);
            }
        const Int4Scale sc = int4_row_scale(low, high, odd, LANES, 0xffffffffu);
        if (slot < 0) continue;
        const int64_t block = slot / a.block_size;
        const int64_t row =
            (block * a.hkv + (r - t * a.hkv)) * a.block_size + (slot - block * a.block_size);
        uint8_t *pool = (is_k ? a.k_pool : a.v_pool) + row * (d / 2);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int e = (c + u * LANES) * 16;
            if (e < d) {
                float x[8];
                unpack8(raw[u][0], x);
                const uint32_t w0 = int4_codes8(x, sc);
                unpack8(raw[u][1], x);
                *reinterpret_cast<uint2 *>(pool + e / 2) = make_uint2(w0, int4_codes8(x, sc));
            }
        }
        if (c == 0) (is_k ? a.k_params : a.v_params)[row] = sc.params;
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
    const int64_t steps = (2 * num_tokens * a.hkv + kThreads / lanes - 1) / (kThreads / lanes);
    const dim3 grid(unsigned(std::min<int64_t>(steps, int64_t(sm_count()) * 8)));
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
