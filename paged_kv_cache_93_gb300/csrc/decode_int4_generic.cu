// decode_int4_generic.cu -- decode attention over a 4-bit cache on CUDA cores, any shape.
//
// Element d of token j's key is s_j c_jd + o_j with the row's scale s_j and offset o_j, so
//     q . K_j = s_j (q . c_j) + o_j sum_d q_d
// and the values' sum splits likewise into sum_j (p_j s_j) c_j and, the same for every
// element, sum_j p_j o_j: the codes go into the products as numbers and scales and offsets
// are applied once a token.  The numbers are c - 8 (and the offsets o + 8 s): sums of the
// codes themselves would grow with the context and cancel against the offsets'.
//
// One warp per (sequence, query token, split, up to R query heads of a KV head), which
// share what is loaded and taken apart.  W lanes have a row in words of 8 codes (all 32 for
// rows of more than 16 words), so that a warp reads 32 / W sets of kU tokens at a time,
// each set with an online softmax (running max m, running sum l) of its own, in base 2
// with the query pre-multiplied by scale * log2(e); the sets are joined at the end.
//
// Bound: instructions, four to six an element and query head.  8 x 32K, 8 KV heads: 32
// query heads of 128 478 us, of 96 507, of 256 1,029, 8 of 96 276 (a head a warp, its row in
// 16 of 32 lanes, codes by conversions and tokens by 64-bit divisions: 3,038, 2,946, 3,290).
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

// The e-th code of a word, less 8: in the low bits of 2^23 it is 2^23 + code.  (Conversions
// run at an eighth of the rate.)
__device__ __forceinline__ float centred(uint32_t word, int e) {
    return __uint_as_float(0x4b000000u | ((word >> (4 * e)) & 15u)) - 8388616.f;
}

__device__ __forceinline__ float sum_over(float v, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// C: words of a row that a lane holds (W = 32; otherwise 1).
template <int C, int W, int R>
__global__ void __launch_bounds__(kWarps * 32) decode_int4_generic_kernel(const Int4DecodeArgs a) {
    static_assert(C == 1 || W == 32, "a narrow row is one word a lane");
    constexpr int kStep = kU * (32 / W);
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, part = lane & (W - 1);
    const pkv_cache_desc &c = a.cache;
    const int tiles = (a.group + R - 1) / R;     // of a KV head's query heads
    const int unit = blockIdx.y * kWarps + (threadIdx.x >> 5);
    const int g = unit / tiles, first = (unit - g * tiles) * R, h0 = g * a.group + first;
    const int row = blockIdx.z;                  // sequence-major: b * T + t
    const int b = row / a.q_tokens, t = row - b * a.q_tokens;
    const int split = blockIdx.x;
    if (g >= c.num_kv_heads) return;
    const int nk = c.head_dim_k / 8, nv = c.head_dim_v / 8;
    const bool tells = lane == 0 && first == 0;

    int64_t L = a.seq_lens[b];
    const bool odd = L < 0 || L > int64_t(a.max_blocks) * c.block_size;
    if ((odd || L < a.flag_below) && tells && split == 0 && t == 0)
        raise_status(a.status, PKV_DEV_SEQ_LEN);
    if (odd) L = 0;
    const int64_t chunk = 64 * ((L + 64LL * a.num_splits - 1) / (64LL * a.num_splits));
    const int64_t begin = int64_t(split) * chunk;
    const int64_t seen = L - a.q_tokens + 1 + t;        // tokens that this row sees
    const int64_t end = seen < begin + chunk ? seen : begin + chunk;

    // the queries, pre-scaled so that scores come out in base-2 log units, and their sums
    float qv[R][C][8], qsum[R];
    const float qscale = a.scale * kLog2e;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = first + r < a.group;
        const float *qrow = a.q + (int64_t(row) * a.num_q_heads + h0 + (in ? r : 0)) * c.head_dim_k;
        qsum[r] = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int v = part + W * i;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                qv[r][i][e] = in && v < nk ? qrow[v * 8 + e] * qscale : 0.f;
                qsum[r] += qv[r][i][e];
            }
        }
        qsum[r] = sum_over(qsum[r], W);
    }
    float acc[R][C][8], m[R], l[R], off[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = off[r] = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[r][i][e] = 0.f;
    }

    const int32_t *table = a.block_tables + int64_t(b) * a.max_blocks;
    for (int64_t at0 = begin; at0 < end; at0 += kStep) {
        // this set's tokens j0 .. j0 + kU - 1; those at or past `end` are not seen.  A
        // block id out of range is flagged and its token reads as zeros.
        const int64_t j0 = at0 + lane / W * kU;
        int64_t at[kU];
        bool live[kU], ok[kU];
        uint32_t kp[kU], vp[kU];
        uint32_t block = uint32_t(j0) / uint32_t(c.block_size);      // (lengths are 32-bit)
        int32_t place = int32_t(uint32_t(j0) - block * uint32_t(c.block_size));
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            live[u] = j0 + u < end;
            const int32_t phys = live[u] ? table[block] : 0;
            ok[u] = live[u] && phys >= 0 && phys < c.num_blocks;
            if (live[u] && !ok[u] && part == 0 && first == 0)
                raise_status(a.status, PKV_DEV_BLOCK_ID);
            at[u] = (int64_t(ok[u] ? phys : 0) * c.num_kv_heads + g) * c.block_size + place;
            if (++place == c.block_size) {
                place = 0;
                ++block;
            }
            kp[u] = ok[u] ? a.k_params[at[u]] : 0u;
            vp[u] = ok[u] ? a.v_params[at[u]] : 0u;
        }
        uint32_t kr[kU][C], vr[kU][C];
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int v = part + W * i;
                const uint32_t *k = reinterpret_cast<const uint32_t *>(a.k_pool) + at[u] * nk;
                const uint32_t *x = reinterpret_cast<const uint32_t *>(a.v_pool) + at[u] * nv;
                kr[u][i] = v < nk && ok[u] ? k[v] : 0u;
                vr[u][i] = v < nv && ok[u] ? x[v] : 0u;
            }
        float sc[kU][R];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
#pragma unroll
            for (int r = 0; r < R; ++r) sc[u][r] = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float k = centred(kr[u][i], e);
#pragma unroll
                    for (int r = 0; r < R; ++r) sc[u][r] = fmaf(qv[r][i][e], k, sc[u][r]);
                }
        }
        float w[kU][R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float m_new = m[r];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const float dot = sum_over(sc[u][r], W), ks = bf16_lo_to_f32(kp[u]);
                sc[u][r] = live[u] ? fmaf(ks, dot, fmaf(ks, 8.f, bf16_hi_to_f32(kp[u])) * qsum[r])
                                   : -INFINITY;
                m_new = fmaxf(m_new, sc[u][r]);
            }
            const float base = m_new == -INFINITY ? 0.f : m_new;
            const float corr = exp2f(m[r] - base);
            float psum = 0.f, posum = 0.f;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const float p = exp2f(sc[u][r] - base), vs = bf16_lo_to_f32(vp[u]);
                psum += p;
                w[u][r] = live[u] ? p * vs : 0.f;
                posum += live[u] ? p * fmaf(vs, 8.f, bf16_hi_to_f32(vp[u])) : 0.f;
            }
            l[r] = l[r] * corr + psum;
            off[r] = off[r] * corr + posum;
            m[r] = m_new;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[r][i][e] *= corr;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = centred(vr[u][i], e);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[r][i][e] = fmaf(w[u][r], x, acc[r][i][e]);
                }
    }

#pragma unroll
    for (int r = 0; r < R; ++r) {
        // the sets together
        for (int o = W; o < 32; o <<= 1) {
            const float m_other = __shfl_xor_sync(0xffffffffu, m[r], o);
            const float m_new = fmaxf(m[r], m_other), base = m_new == -INFINITY ? 0.f : m_new;
            const float mine = exp2f(m[r] - base), other = exp2f(m_other - base);
            m[r] = m_new;
            l[r] = l[r] * mine + __shfl_xor_sync(0xffffffffu, l[r], o) * other;
            off[r] = off[r] * mine + __shfl_xor_sync(0xffffffffu, off[r], o) * other;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[r][i][e] = acc[r][i][e] * mine +
                                   __shfl_xor_sync(0xffffffffu, acc[r][i][e], o) * other;
        }
        if (first + r >= a.group) continue;
        // (l != l: a row with a NaN score is NaN, sum and output)
        const bool some = l[r] > 0.f || l[r] != l[r];
        const int64_t orow =
            (int64_t(split) * a.batch * a.q_tokens + row) * a.num_q_heads + h0 + r;
        const float inv = some ? 1.f / l[r] : 0.f;
        float *o = a.out_part + orow * c.head_dim_v;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int v = part + W * i;
            if (lane < W && v < nv) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = some ? (acc[r][i][e] + off[r]) * inv : 0.f;
                reinterpret_cast<float4 *>(o)[2 * v] = make_float4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<float4 *>(o)[2 * v + 1] = make_float4(y[4], y[5], y[6], y[7]);
            }
        }
        if (lane == 0) a.lse_part[orow] = some ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
    }
}

// Query heads of a warp: four share a row's codes where registers hold them (8 x 32K, 8 KV
// heads of 96, two query heads each: 505 us, one each 276; alone on a warp twice that).
int rows_of(const pkv_cache_desc &c, int group) {
    return group > 1 && std::max(c.head_dim_k, c.head_dim_v) <= 256 ? 4 : 1;
}

template <int C, int W, int R>
int launch(const Int4DecodeArgs &a) {
    const int64_t units = int64_t(a.cache.num_kv_heads) * ((a.group + R - 1) / R);
    const dim3 grid(a.num_splits, unsigned((units + kWarps - 1) / kWarps), a.batch * a.q_tokens);
    return launch_pdl(decode_int4_generic_kernel<C, W, R>, grid, dim3(kWarps * 32), 0, a.stream,
                      a);
}

}  // namespace

int64_t int4_generic_ctas(const pkv_cache_desc &c, int32_t batch, int32_t num_q_heads,
                          int32_t q_tokens) {
    const int group = num_q_heads / c.num_kv_heads, rows = rows_of(c, group);
    const int64_t units = int64_t(c.num_kv_heads) * ((group + rows - 1) / rows);
    return (units + kWarps - 1) / kWarps * batch * q_tokens;
}

int launch_decode_int4_generic(const Int4DecodeArgs &a) {
    const int words = std::max(a.cache.head_dim_k, a.cache.head_dim_v) / 8;
    if (rows_of(a.cache, a.group) == 4)
        return words <= 8    ? launch<1, 8, 4>(a)
               : words <= 16 ? launch<1, 16, 4>(a)
                             : launch<1, 32, 4>(a);
    return words <= 8    ? launch<1, 8, 1>(a)
           : words <= 16 ? launch<1, 16, 1>(a)
           : words <= 32 ? launch<1, 32, 1>(a)
           : words <= 64 ? launch<2, 32, 1>(a)
                         : launch<4, 32, 1>(a);
}

}  // namespace pkv
