// int4_api.cu -- C ABI entry points of decode attention over a 4-bit cache: argument
// validation, split selection, kernel choice and the split -> merge sequence.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_host.h"

using namespace pkv;

namespace {

constexpr int32_t kMaxSplits = 256;
constexpr int32_t kMaxQueryTokens = 64;
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Whether the tensor-core kernel takes the call.
bool on_tensor_cores(const pkv_cache_desc &c, int32_t batch, int32_t tokens, int32_t hq,
                     int32_t max_blocks, int32_t flags) {
    return !(flags & PKV_DECODE_GENERIC) && hq % c.num_kv_heads == 0 &&
           int4_kernel_supports(c, batch, hq, tokens, max_blocks);
}

// How a call runs: the library's own plan (S = 0), or S chunks, and its workspace.
struct Plan {
    int32_t splits;
    size_t bytes;
};

Plan plan_of(const pkv_cache_desc &c, int32_t batch, int32_t tokens, int32_t hq,
             int32_t max_blocks, int32_t num_splits, int32_t flags) {
    int32_t S = num_splits;
    if (S == 0 && on_tensor_cores(c, batch, tokens, hq, max_blocks, flags)) {
        const size_t bytes = int4_plan_workspace(c, batch, hq, tokens, max_blocks);
        if (bytes) return {0, bytes};
        S = 1;
    }
    if (S == 0) {
        // Eight CTAs an SM, of sequences as long as their table rows 512 tokens each.
        const int64_t ctas = std::max<int64_t>(1, int4_generic_ctas(c, batch, hq, tokens));
        const int64_t want = (int64_t(sm_count()) * 8 + ctas - 1) / ctas;
        const int64_t most = (int64_t(max_blocks) * c.block_size + 511) / 512;
        S = int32_t(std::max<int64_t>(1, std::min<int64_t>({want, most, 64})));
    }
    return {S, pkv_decode_workspace_size(batch * tokens, hq, c.head_dim_v, S)};
}

int run_split_kernel(const Int4DecodeArgs &a, int32_t flags) {
    return on_tensor_cores(a.cache, a.batch, a.q_tokens, a.num_q_heads, a.max_blocks, flags)
               ? launch_decode_int4(a, nullptr)
               : launch_decode_int4_generic(a);
}

// The checks that the entry points share.
int validate(const pkv_cache_desc *c, const float *q, int32_t batch, int32_t tokens, int32_t hq,
             const void *k_pool, const void *k_params, const void *v_pool, const void *v_params,
             const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens,
             int32_t num_splits, int32_t flags, const float *out, const float *lse) {
    const int st = validate_int4_cache(c);
    if (st == PKV_ERR_INVALID_ARG) return st;
    if (batch < 0 || tokens < 1 || tokens > kMaxQueryTokens || hq <= 0 || max_blocks < 0 ||
        num_splits < 0 || num_splits > kMaxSplits ||
        (flags & ~(PKV_DECODE_GENERIC | PKV_DECODE_NO_TCGEN05)) != 0)
        return PKV_ERR_INVALID_ARG;
    if (st != PKV_OK || hq % c->num_kv_heads != 0 || int64_t(batch) * tokens > 65535)
        return PKV_ERR_SHAPE;
    // the generic kernel's grid
    if (hq > 4 * 65535) return PKV_ERR_SHAPE;
    if (batch == 0) return PKV_OK;
    if (!q || !k_pool || !k_params || !v_pool || !v_params || !block_tables || !seq_lens ||
        !out || !lse)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pool) || !aligned16(k_params) || !aligned16(v_pool) ||
        !aligned16(v_params) || !aligned16(out))
        return PKV_ERR_ALIGNMENT;
    return PKV_OK;
}

Int4DecodeArgs args_of(const pkv_cache_desc *c, const float *q, int32_t batch, int32_t tokens,
                       int32_t hq, const void *k_pool, const void *k_params, const void *v_pool,
                       const void *v_params, const int32_t *block_tables, int32_t max_blocks,
                       const int32_t *seq_lens, float scale, int32_t splits, float *out_part,
                       float *lse_part, int32_t flag_below, pkv_stream_t stream) {
    Int4DecodeArgs a = {};
    a.cache = *c;
    a.q = q;
    a.batch = batch;
    a.q_tokens = tokens;
    a.num_q_heads = hq;
    a.group = hq / c->num_kv_heads;
    a.k_pool = static_cast<const uint8_t *>(k_pool);
    a.v_pool = static_cast<const uint8_t *>(v_pool);
    a.k_params = static_cast<const uint32_t *>(k_params);
    a.v_params = static_cast<const uint32_t *>(v_params);
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.scale = scale;
    a.num_splits = splits;
    a.out_part = out_part;
    a.lse_part = lse_part;
    a.flag_below = flag_below;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    return a;
}

int attend(const pkv_cache_desc *cache, const float *q, int32_t batch, int32_t tokens,
           int32_t hq, const void *k_pool, const void *k_params, const void *v_pool,
           const void *v_params, const int32_t *block_tables, int32_t max_blocks,
           const int32_t *seq_lens, float scale, int32_t num_splits, void *workspace,
           size_t workspace_bytes, float *out, float *lse, int32_t flag_below, int32_t flags,
           pkv_stream_t stream) {
    int st = validate(cache, q, batch, tokens, hq, k_pool, k_params, v_pool, v_params,
                      block_tables, max_blocks, seq_lens, num_splits, flags, out, lse);
    if (st != PKV_OK || batch == 0) return st;
    const int32_t rows = batch * tokens;
    const Plan plan = plan_of(*cache, batch, tokens, hq, max_blocks, num_splits, flags);
    const int32_t S = plan.splits;
    if (plan.bytes && (!workspace || workspace_bytes < plan.bytes))
        return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (plan.bytes && !aligned16(workspace)) return PKV_ERR_ALIGNMENT;
    Int4DecodeArgs a =
        args_of(cache, q, batch, tokens, hq, k_pool, k_params, v_pool, v_params, block_tables,
                max_blocks, seq_lens, scale, S, out, lse, flag_below, stream);
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    if (S == 0) return launch_decode_int4(a, workspace);
    if (S == 1) return run_split_kernel(a, flags);
    const size_t parts = size_t(S) * rows * hq;
    char *ws = static_cast<char *>(workspace);
    a.out_part = reinterpret_cast<float *>(ws);
    a.lse_part =
        reinterpret_cast<float *>(ws + align256(parts * cache->head_dim_v * sizeof(float)));
    st = run_split_kernel(a, flags);
    if (st != PKV_OK) return st;
    return launch_lse_merge(S, a.out_part, a.lse_part, int64_t(rows) * hq, cache->head_dim_v, out,
                            lse, a.stream);
}

}  // namespace

extern "C" size_t pkv_decode_workspace_size_int4(const pkv_cache_desc *cache, int32_t batch,
                                                 int32_t tokens_per_seq, int32_t num_q_heads,
                                                 int32_t max_blocks, int32_t num_splits,
                                                 int32_t flags) {
    if (validate_int4_cache(cache) != PKV_OK || batch <= 0 || tokens_per_seq < 1 ||
        tokens_per_seq > kMaxQueryTokens || num_q_heads <= 0 || max_blocks < 0 ||
        num_splits < 0 || num_splits > kMaxSplits || num_q_heads % cache->num_kv_heads != 0 ||
        int64_t(batch) * tokens_per_seq > 65535)
        return 0;
    return plan_of(*cache, batch, tokens_per_seq, num_q_heads, max_blocks, num_splits, flags).bytes;
}

extern "C" int pkv_paged_decode_attn_int4(
    const pkv_cache_desc *cache, const float *q, int32_t batch, int32_t num_q_heads,
    const void *k_pool, const void *k_params, const void *v_pool, const void *v_params,
    const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens, float scale,
    int32_t num_splits, void *workspace, size_t workspace_bytes, float *out, float *lse,
    int32_t flags, pkv_stream_t stream) {
    return attend(cache, q, batch, 1, num_q_heads, k_pool, k_params, v_pool, v_params,
                  block_tables, max_blocks, seq_lens, scale, num_splits, workspace,
                  workspace_bytes, out, lse, 0, flags, stream);
}

extern "C" int pkv_paged_decode_attn_multi_int4(
    const pkv_cache_desc *cache, const float *q, int32_t batch, int32_t tokens_per_seq,
    int32_t num_q_heads, const void *k_pool, const void *k_params, const void *v_pool,
    const void *v_params, const int32_t *block_tables, int32_t max_blocks,
    const int32_t *seq_lens, float scale, int32_t num_splits, void *workspace,
    size_t workspace_bytes, float *out, float *lse, int32_t flags, pkv_stream_t stream) {
    return attend(cache, q, batch, tokens_per_seq, num_q_heads, k_pool, k_params, v_pool,
                  v_params, block_tables, max_blocks, seq_lens, scale, num_splits, workspace,
                  workspace_bytes, out, lse, tokens_per_seq, flags, stream);
}

extern "C" int pkv_paged_decode_attn_partial_int4(
    const pkv_cache_desc *cache, const float *q, int32_t batch, int32_t num_q_heads,
    const void *k_pool, const void *k_params, const void *v_pool, const void *v_params,
    const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens, float scale,
    int32_t num_splits, float *out_part, float *lse_part, int32_t flags, pkv_stream_t stream) {
    const int st =
        validate(cache, q, batch, 1, num_q_heads, k_pool, k_params, v_pool, v_params,
                 block_tables, max_blocks, seq_lens, num_splits, flags, out_part, lse_part);
    if (st != PKV_OK || batch == 0) return st;
    if (num_splits < 1) return PKV_ERR_INVALID_ARG;
    Int4DecodeArgs a = args_of(cache, q, batch, 1, num_q_heads, k_pool, k_params, v_pool,
                               v_params, block_tables, max_blocks, seq_lens, scale, num_splits,
                               out_part, lse_part, 0, stream);
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    return run_split_kernel(a, flags);
}
