// decode_int4_generic.cu -- decode attention over a 4-bit cache on CUDA cores, any shape.
//
// Element d of token j's key is s_j c_jd + o_j with the row's scale s_j and offset o_j, so
//     q . K_j = s_j (q . c_j) + o_j sum_d q_d
// and the values' sum splits likewise into sum_j (p_j s_j) c_j and, the same for every
// element, sum_j p_j o_j: the codes go into the products as numbers and scales and offsets
// are applied once a token.  The numbers are c - 7.5 (and the offsets o + 7.5 s): sums of
// the codes themselves would grow with the context and cancel against the offsets'.
//
// One warp per (sequence, query token, query head, split); lanes split a row into words
// of 8 codes, a token's score is a warp reduction, and the online softmax (running max
// m, running sum l) runs in base 2 with the query pre-multiplied by scale * log2(e).  A
// warp takes kU tokens per step, so that as many rows are on their way.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;
constexpr int kU = 4;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The e-th code of a word, less 7.5.
__device__ __forceinline__ float centred(uint32_t word, int e) {
    return float((word >> (4 * e)) & 15u) - 7.5f;
}

// KC / VC: words of a K and of a V row a lane holds (ceil(dim / 256)).
template <int KC, int VC>
__global__ void __launch_bounds__(kWarps * 32) decode_int4_generic_kernel(const Int4DecodeArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * kWarps + (threadIdx.x >> 5);
    const int row = blockIdx.z;                  // sequence-major: b * T + t
    const int b = row / a.q_tokens, t = row - b * a.q_tokens;
    const int split = blockIdx.x;
    if (h >= a.num_q_heads) return;
    const pkv_cache_desc &c = a.cache;
    const int group = a.num_q_heads / c.num_kv_heads;
    const int g = h / group;
    const int nk = c.head_dim_k / 8, nv = c.head_dim_v / 8;

    int64_t L = a.seq_lens[b];
    const bool odd = L < 0 || L > int64_t(a.max_blocks) * c.block_size;
    if ((odd || L < a.flag_below) && lane == 0 && split == 0 && t == 0 && h % group == 0)
        raise_status(a.status, PKV_DEV_SEQ_LEN);
    if (odd) L = 0;
    const int64_t chunk = 64 * ((L + 64LL * a.num_splits - 1) / (64LL * a.num_splits));
    const int64_t begin = int64_t(split) * chunk;
    const int64_t seen = L - a.q_tokens + 1 + t;        // tokens that this row sees
    const int64_t end = seen < begin + chunk ? seen : begin + chunk;

    // q, pre-scaled so that scores come out in base-2 log units, and its sum
    float qv[KC][8], qsum = 0.f;
    const float qscale = a.scale * kLog2e;
    const float *qrow = a.q + (int64_t(row) * a.num_q_heads + h) * c.head_dim_k;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const int v = lane + 32 * i;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            qv[i][e] = v < nk ? qrow[v * 8 + e] * qscale : 0.f;
            qsum += qv[i][e];
        }
    }
    qsum = warp_sum(qsum);
    float acc[VC][8];
#pragma unroll
    for (int i = 0; i < VC; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
    float m = -INFINITY, l = 0.f, off = 0.f;

    const int32_t *table = a.block_tables + int64_t(b) * a.max_blocks;
    for (int64_t j0 = begin; j0 < end; j0 += kU) {
        // tokens j0 .. j0 + kU - 1; those at or past `end` are not seen.  A block id out
        // of range is flagged and its token reads as zeros.
        int64_t at[kU];
        bool live[kU], ok[kU];
        uint32_t kp[kU], vp[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t j = j0 + u;
            live[u] = j < end;
            const int32_t phys = live[u] ? table[j / c.block_size] : 0;
            ok[u] = live[u] && phys >= 0 && phys < c.num_blocks;
            if (live[u] && !ok[u] && lane == 0 && h % group == 0)
                raise_status(a.status, PKV_DEV_BLOCK_ID);
            at[u] = (int64_t(ok[u] ? phys : 0) * c.num_kv_heads + g) * c.block_size +
                    j % c.block_size;
            kp[u] = ok[u] ? a.k_params[at[u]] : 0u;
            vp[u] = ok[u] ? a.v_params[at[u]] : 0u;
        }
        uint32_t kr[kU][KC];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const int v = lane + 32 * i;
                kr[u][i] = v < nk && ok[u]
                               ? reinterpret_cast<const uint32_t *>(a.k_pool)[at[u] * nk + v]
                               : 0u;
            }
        float sc[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < KC; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    part = fmaf(qv[i][e], centred(kr[u][i], e), part);
            sc[u] = part;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const float dot = warp_sum(sc[u]);
            const float ks = bf16_lo_to_f32(kp[u]);
            sc[u] = live[u] ? fmaf(ks, dot, fmaf(ks, 7.5f, bf16_hi_to_f32(kp[u])) * qsum)
                            : -INFINITY;
        }
        float m_new = m;
#pragma unroll
        for (int u = 0; u < kU; ++u) m_new = fmaxf(m_new, sc[u]);
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float corr = exp2f(m - base);
        float w[kU], psum = 0.f, posum = 0.f;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const float p = exp2f(sc[u] - base);
            psum += p;
            w[u] = live[u] ? p * bf16_lo_to_f32(vp[u]) : 0.f;
            posum += live[u] ? p * fmaf(bf16_lo_to_f32(vp[u]), 7.5f, bf16_hi_to_f32(vp[u])) : 0.f;
        }
        l = l * corr + psum;
        off = off * corr + posum;
        m = m_new;
        uint32_t vr[kU][VC];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < VC; ++i) {
                const int v = lane + 32 * i;
                vr[u][i] = v < nv && ok[u]
                               ? reinterpret_cast<const uint32_t *>(a.v_pool)[at[u] * nv + v]
                               : 0u;
            }
#pragma unroll
        for (int i = 0; i < VC; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[i][e] *= corr;
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    acc[i][e] = fmaf(w[u], centred(vr[u][i], e), acc[i][e]);
            }
    }

    // (l != l: a row with a NaN score is NaN, sum and output)
    const bool some = l > 0.f || l != l;
    const int64_t orow =
        (int64_t(split) * a.batch * a.q_tokens + row) * a.num_q_heads + h;
    const float inv = some ? 1.f / l : 0.f;
    float *o = a.out_part + orow * c.head_dim_v;
#pragma unroll
    for (int i = 0; i < VC; ++i) {
        const int v = lane + 32 * i;
        if (v < nv) {
            float r[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = some ? (acc[i][e] + off) * inv : 0.f;
            reinterpret_cast<float4 *>(o)[2 * v] = make_float4(r[0], r[1], r[2], r[3]);
            reinterpret_cast<float4 *>(o)[2 * v + 1] = make_float4(r[4], r[5], r[6], r[7]);
        }
    }
    if (lane == 0) a.lse_part[orow] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <int KC, int VC>
int launch(const Int4DecodeArgs &a) {
    const dim3 grid(a.num_splits, (a.num_q_heads + kWarps - 1) / kWarps, a.batch * a.q_tokens);
    return launch_pdl(decode_int4_generic_kernel<KC, VC>, grid, dim3(kWarps * 32), 0, a.stream,
                      a);
}

}  // namespace

int launch_decode_int4_generic(const Int4DecodeArgs &a) {
    const int kc = (a.cache.head_dim_k + 255) / 256, vc = (a.cache.head_dim_v + 255) / 256;
    const int n = std::max(kc, vc);
    return n == 1 ? launch<1, 1>(a) : n == 2 ? launch<2, 2>(a) : launch<4, 4>(a);
}

}  // namespace pkv
