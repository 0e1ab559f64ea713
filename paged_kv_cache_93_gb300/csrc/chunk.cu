// chunk.cu -- C ABI entry points of the attention of ragged chunks of new
// tokens: argument checks and kernel choice.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "pkv_host.h"

namespace pkv {
namespace {

// (sequence, KV head) pairs up to which the merge counts its pieces in 32 bits: 32 of each
// (128 rows, 4 a piece), 64 of each of the 256 cuts at most, and the grid's stride.
constexpr int64_t kMostPairs = (int64_t(1) << 26) - 2048;

// Whether a call of this shape runs on the tensor cores (which alone read the test
// control).
bool on_tensor_cores(const pkv_cache_desc &c, int64_t num_tokens, int32_t batch, int32_t hq,
                     int32_t max_blocks, int32_t flags, bool e4, bool values_in_keys) {
    return (flags & ~PKV_DECODE_TEST_WITHHOLD) == 0 && !values_in_keys && chunk_tc_supports(c, hq, max_blocks, e4) &&
           std::min<int64_t>(num_tokens, batch) * c.num_kv_heads <= kMostPairs;
}

size_t workspace_size(const pkv_cache_desc *c, int64_t num_tokens, int32_t batch, int32_t hq,
                      int32_t max_blocks, int32_t flags, bool e4) {
    if (!c || num_tokens <= 0 || batch <= 0 || hq <= 0 || max_blocks < 0 ||
        c->num_kv_heads <= 0 || hq % c->num_kv_heads != 0 || c->num_blocks <= 0 ||
        num_tokens >= ((int64_t(1) << 29) + hq - 1) / hq ||
        !on_tensor_cores(*c, num_tokens, batch, hq, max_blocks, flags, e4, false))
        return 0;
    return chunk_tc_workspace(*c, num_tokens, batch, hq);
}

// Runs a checked call.
int run(ChunkArgs &a, bool e4, bool values_in_keys, void *workspace, size_t workspace_bytes,
        int32_t flags) {
    const bool tc = on_tensor_cores(a.cache, a.num_tokens, a.batch, a.num_q_heads, a.max_blocks,
                                    flags, e4, values_in_keys);
    a.withhold = (flags & PKV_DECODE_TEST_WITHHOLD) != 0;
    if (a.withhold && !tc) return PKV_ERR_INVALID_ARG;
    if (tc) {
        const size_t need =
            chunk_tc_workspace(a.cache, a.num_tokens, a.batch, a.num_q_heads);
        if (!workspace || workspace_bytes < need) return PKV_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace)) return PKV_ERR_ALIGNMENT;
    }
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    if (tc) return launch_chunk_tc(a, workspace);
    return e4 ? launch_chunk_generic_e4m3(a) : launch_chunk_generic(a);
}

// The host checks both entry points share; fills all of `a` but the scales.
// *done: nothing to launch.
int prepare(ChunkArgs &a, bool e4, const pkv_cache_desc *c, const void *q, int64_t num_tokens,
            int32_t hq, const int32_t *cu_q_lens, int32_t batch, const void *k_pool,
            const void *v_pool, const int32_t *block_tables, int32_t max_blocks,
            const int32_t *seq_lens, float scale, int32_t window, int32_t sink_tokens, void *out,
            float *lse, int32_t flags, cudaStream_t stream, bool *done) {
    *done = false;
    const int32_t known = PKV_DECODE_GENERIC | PKV_DECODE_NO_TCGEN05 |
                          (test_withhold_enabled() ? PKV_DECODE_TEST_WITHHOLD : 0);
    if (!c || num_tokens < 0 || batch < 0 || hq <= 0 || max_blocks < 0 || window < 0 ||
        sink_tokens < 0 || !(scale > 0.f) || !std::isfinite(scale) || (flags & ~known) != 0)
        return PKV_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->block_size < 1 || c->block_size > 256 || c->num_kv_heads <= 0 ||
        c->head_dim_k <= 0 || c->head_dim_v <= 0)
        return PKV_ERR_INVALID_ARG;
    if (hq % c->num_kv_heads != 0 || c->head_dim_k % 8 != 0 || c->head_dim_v % 8 != 0 ||
        c->head_dim_k > 1024 || c->head_dim_v > 1024 || batch > 65535 || hq > 65535 ||
        num_tokens >= ((int64_t(1) << 29) + hq - 1) / hq)
        return PKV_ERR_SHAPE;
    if (num_tokens == 0 || batch == 0) {
        *done = true;
        return PKV_OK;
    }
    if (!q || !cu_q_lens || !k_pool || !block_tables || !seq_lens || !out || (e4 && !v_pool))
        return PKV_ERR_INVALID_ARG;
    if (!v_pool && c->head_dim_v > c->head_dim_k) return PKV_ERR_SHAPE;   // values inside the keys
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_pool) || (v_pool && !aligned16(v_pool)))
        return PKV_ERR_ALIGNMENT;
    a.cache = *c;
    a.q = q;
    a.num_tokens = int32_t(num_tokens);
    a.batch = batch;
    a.num_q_heads = hq;
    a.cu_q_lens = cu_q_lens;
    a.k_pool = k_pool;
    a.v_pool = v_pool ? v_pool : k_pool;
    a.v_stride = v_pool ? c->head_dim_v : c->head_dim_k;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.scale = scale;
    // no position reaches the table's capacity: a wider window masks nothing, more
    // sinks add none, and the kernels' differences of positions stay in range
    const int64_t capacity = int64_t(max_blocks) * c->block_size;
    a.window = window >= capacity ? 0 : window;
    a.sinks = int32_t(std::min<int64_t>(sink_tokens, capacity));
    a.out = out;
    a.lse = lse;
    a.stream = stream;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_chunk_workspace_size(const pkv_cache_desc *cache, int64_t num_tokens,
                                           int32_t batch, int32_t num_q_heads, int32_t max_blocks,
                                           int32_t flags) {
    return workspace_size(cache, num_tokens, batch, num_q_heads, max_blocks, flags, false);
}

extern "C" size_t pkv_chunk_workspace_size_e4m3(const pkv_cache_desc *cache, int64_t num_tokens,
                                                int32_t batch, int32_t num_q_heads,
                                                int32_t max_blocks, int32_t flags) {
    return workspace_size(cache, num_tokens, batch, num_q_heads, max_blocks, flags, true);
}

extern "C" int pkv_paged_chunk_attn(const pkv_cache_desc *cache, const void *q,
                                    int64_t num_tokens, int32_t num_q_heads,
                                    const int32_t *cu_q_lens, int32_t batch, const void *k_pool,
                                    const void *v_pool, const int32_t *block_tables,
                                    int32_t max_blocks, const int32_t *seq_lens, float scale,
                                    int32_t window, int32_t sink_tokens, void *workspace,
                                    size_t workspace_bytes, void *out, float *lse, int32_t flags,
                                    pkv_stream_t stream) {
    ChunkArgs a = {};
    bool done;
    const int rc = prepare(a, false, cache, q, num_tokens, num_q_heads, cu_q_lens, batch, k_pool,
                           v_pool, block_tables, max_blocks, seq_lens, scale, window, sink_tokens,
                           out, lse, flags, reinterpret_cast<cudaStream_t>(stream), &done);
    if (rc != PKV_OK || done) return rc;
    return run(a, false, !v_pool, workspace, workspace_bytes, flags);
}

extern "C" int pkv_paged_chunk_attn_e4m3(const pkv_cache_desc *cache, const void *q,
                                         int64_t num_tokens, int32_t num_q_heads,
                                         const int32_t *cu_q_lens, int32_t batch,
                                         const void *k_pool, const void *v_pool,
                                         const float *k_scale, const float *v_scale,
                                         const int32_t *block_tables, int32_t max_blocks,
                                         const int32_t *seq_lens, float scale, int32_t window,
                                         int32_t sink_tokens, void *workspace,
                                         size_t workspace_bytes, void *out, float *lse,
                                         int32_t flags, pkv_stream_t stream) {
    ChunkArgs a = {};
    bool done;
    const int rc = prepare(a, true, cache, q, num_tokens, num_q_heads, cu_q_lens, batch, k_pool,
                           v_pool, block_tables, max_blocks, seq_lens, scale, window, sink_tokens,
                           out, lse, flags, reinterpret_cast<cudaStream_t>(stream), &done);
    if (rc != PKV_OK || done) return rc;
    if (!k_scale || !v_scale) return PKV_ERR_INVALID_ARG;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    return run(a, true, false, workspace, workspace_bytes, flags);
}
