// chunk_generic.cu -- attention of ragged chunks of new tokens over the paged
// cache on CUDA cores: any head dims (multiples of 8 up to 1024), any query
// group, any block size, values inside the keys, bf16 or E4M3 pools.
//
// One CTA per (token, up to kHeads query heads of one KV head).  Its warps
// take every kWarps-th group of kU keys the token sees; lanes split the head
// dimension into 8-element vectors, each K and V row is loaded once for the
// CTA's heads, and the online softmax (running max, running sum, rescaled
// accumulator, base 2) is kept per head and warp in fp32, joined through
// shared memory at the end.  Keys a token does not see are never loaded, so
// nothing they hold reaches the result.  Bound by its fp32 arithmetic: the
// tensor-core kernel takes the common shapes.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 4;
constexpr int kHeads = 4;
constexpr int kU = 2;                   // keys per step of a warp

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    f[0] = bf16_lo_to_f32(u.x); f[1] = bf16_hi_to_f32(u.x);
    f[2] = bf16_lo_to_f32(u.y); f[3] = bf16_hi_to_f32(u.y);
    f[4] = bf16_lo_to_f32(u.z); f[5] = bf16_hi_to_f32(u.z);
    f[6] = bf16_lo_to_f32(u.w); f[7] = bf16_hi_to_f32(u.w);
}
__device__ __forceinline__ void unpack8(const uint2 &u, float (&f)[8]) {
    const float2 a = e4m3x2_to_f32(u.x & 0xffffu), b = e4m3x2_to_f32(u.x >> 16);
    const float2 c = e4m3x2_to_f32(u.y & 0xffffu), d = e4m3x2_to_f32(u.y >> 16);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}
template <bool E4>
using Raw8 = typename std::conditional<E4, uint2, uint4>::type;

// The sequence whose rows hold token t: the last b with cu[b] <= t (empty
// sequences skipped), or -1 when t is padding.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int batch, int t) {
    int lo = 0, hi = batch;             // cu[lo] <= t < cu[hi] is sought
    if (batch == 0 || t < cu[0] || t >= cu[batch]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// KC / VC: 8-element groups per lane for K and V (ceil(dim / 8 / 32)).
template <int KC, int VC, bool E4>
__global__ void __launch_bounds__(kWarps * 32)
chunk_generic_kernel(const ChunkArgs a) {
    extern __shared__ float joined[];   // [warp][head](dv + 2)
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const pkv_cache_desc &c = a.cache;
    const int t = blockIdx.x;
    const int group = a.num_q_heads / c.num_kv_heads;
    const int parts = (group + kHeads - 1) / kHeads;
    const int g = blockIdx.y / parts, h0 = (blockIdx.y % parts) * kHeads;
    const int nh = min(kHeads, group - h0);
    const bool reporter = blockIdx.y == 0 && threadIdx.x == 0;
    if (t == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b <= a.batch; b += kWarps * 32) {
            const int x = a.cu_q_lens[b];
            if (x < 0 || x > a.num_tokens || (b > 0 && a.cu_q_lens[b - 1] > x))
                raise_status(a.status, PKV_DEV_QUERY_RANGE);
            // (of a sequence with new tokens its own CTAs tell)
            const int L = b < a.batch ? a.seq_lens[b] : 0;
            if (L < 0 || L > int64_t(a.max_blocks) * c.block_size)
                raise_status(a.status, PKV_DEV_SEQ_LEN);
        }
    const int b = sequence_of(a.cu_q_lens, a.batch, t);
    if (b < 0) return;
    const int first = a.cu_q_lens[b], n = a.cu_q_lens[b + 1] - first;
    int64_t L = a.seq_lens[b];
    if (L < 0 || L > int64_t(a.max_blocks) * c.block_size) {
        if (reporter) raise_status(a.status, PKV_DEV_SEQ_LEN);
        L = 0;
    } else if (L < n && reporter) {
        raise_status(a.status, PKV_DEV_SEQ_LEN);
    }
    // The keys this token sees: [0, s) and [w, p + 1), as one run of s +
    // (p + 1 - w) of them.
    const int64_t p = L - n + (t - first);
    int64_t w = a.window > 0 ? p - a.window + 1 : 0;
    if (w < 0) w = 0;
    int64_t s = a.sinks < w ? a.sinks : w;
    const int64_t seen = p >= 0 && p < L ? s + (p + 1 - w) : 0;

    const int nk = c.head_dim_k / 8, nv = c.head_dim_v / 8, vs = a.v_stride / 8;
    const float qscale = a.scale * kLog2e * (E4 ? a.k_scale[g] : 1.f);
    float qv[kHeads][KC][8], acc[kHeads][VC][8], m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        const uint4 *qrow = static_cast<const uint4 *>(a.q) +
                            (int64_t(t) * a.num_q_heads + g * group + h0 + min(h, nh - 1)) * nk;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const int v = lane + 32 * i;
            unpack8(v < nk ? qrow[v] : make_uint4(0, 0, 0, 0), qv[h][i]);
#pragma unroll
            for (int e = 0; e < 8; ++e) qv[h][i][e] *= qscale;
        }
#pragma unroll
        for (int i = 0; i < VC; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[h][i][e] = 0.f;
        m[h] = -INFINITY;
        l[h] = 0.f;
    }
    const int32_t *table = a.block_tables + int64_t(b) * a.max_blocks;
    for (int64_t j0 = int64_t(warp) * kU; j0 < seen; j0 += kWarps * kU) {
        int64_t row[kU];
        bool ok[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            int64_t j = j0 + u;
            ok[u] = j < seen;
            if (!ok[u]) j = 0;
            if (j >= s) j += w - s;
            if (!ok[u]) j = 0;
            int32_t phys = ok[u] ? table[j / c.block_size] : 0;
            if (phys < 0 || phys >= c.num_blocks) {
                if (lane == 0) raise_status(a.status, PKV_DEV_BLOCK_ID);
                phys = 0;
            }
            row[u] = (int64_t(phys) * c.num_kv_heads + g) * c.block_size + j % c.block_size;
        }
        Raw8<E4> kr[kU][KC], vr[kU][VC];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const int v = lane + 32 * i;
                kr[u][i] = v < nk && ok[u]
                               ? static_cast<const Raw8<E4> *>(a.k_pool)[row[u] * nk + v]
                               : Raw8<E4>{};
            }
#pragma unroll
            for (int i = 0; i < VC; ++i) {
                const int v = lane + 32 * i;
                vr[u][i] = v < nv && ok[u]
                               ? static_cast<const Raw8<E4> *>(a.v_pool)[row[u] * vs + v]
                               : Raw8<E4>{};
            }
        }
        float sc[kU][kHeads];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float part[kHeads] = {};
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                float kf[8];
                unpack8(kr[u][i], kf);
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
#pragma unroll
                    for (int e = 0; e < 8; ++e) part[h] = fmaf(qv[h][i][e], kf[e], part[h]);
            }
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
                sc[u][h] = ok[u] ? warp_sum(part[h]) : -INFINITY;
        }
        float pr[kU][kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            float mx = m[h];
#pragma unroll
            for (int u = 0; u < kU; ++u) mx = fmaxf(mx, sc[u][h]);
            const float base = mx == -INFINITY ? 0.f : mx;
            const float corr = exp2f(m[h] - base);
            m[h] = mx;
            l[h] *= corr;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                pr[u][h] = exp2f(sc[u][h] - base);
                l[h] += pr[u][h];
            }
#pragma unroll
            for (int i = 0; i < VC; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[h][i][e] *= corr;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int i = 0; i < VC; ++i) {
                float vf[8];
                unpack8(vr[u][i], vf);
#pragma unroll
                for (int h = 0; h < kHeads; ++h)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[h][i][e] = fmaf(pr[u][h], vf[e], acc[h][i][e]);
            }
    }

    // ---- join the warps
    const int stride = c.head_dim_v + 2;
    float *mine = joined + warp * kHeads * stride;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (lane == 0) {
            mine[h * stride + c.head_dim_v] = m[h];
            mine[h * stride + c.head_dim_v + 1] = l[h];
        }
#pragma unroll
        for (int i = 0; i < VC; ++i) {
            const int v = lane + 32 * i;
            if (v < nv)
#pragma unroll
                for (int e = 0; e < 8; ++e) mine[h * stride + v * 8 + e] = acc[h][i][e];
        }
    }
    __syncthreads();
    const float vscale = E4 ? a.v_scale[g] : 1.f;
    for (int idx = threadIdx.x; idx < nh * c.head_dim_v; idx += kWarps * 32) {
        const int h = idx / c.head_dim_v, d = idx - h * c.head_dim_v;
        float mx = -INFINITY;
        for (int x = 0; x < kWarps; ++x)
            mx = fmaxf(mx, joined[(x * kHeads + h) * stride + c.head_dim_v]);
        // (scores that are all NaN leave no maximum, but a sum that is NaN)
        const float base = mx == -INFINITY ? 0.f : mx;
        float o = 0.f, sum = 0.f;
        for (int x = 0; x < kWarps; ++x) {
            const float *part = joined + (x * kHeads + h) * stride;
            const float wt = exp2f(part[c.head_dim_v] - base);
            sum = fmaf(wt, part[c.head_dim_v + 1], sum);
            o = fmaf(wt, part[d], o);
        }
        const int64_t orow = int64_t(t) * a.num_q_heads + g * group + h0 + h;
        const bool empty = sum == 0.f;
        static_cast<uint16_t *>(a.out)[orow * c.head_dim_v + d] =
            uint16_t(f32_to_bf16_bits(empty ? 0.f : o * vscale / sum));
        if (d == 0 && a.lse) a.lse[orow] = empty ? -INFINITY : (mx + log2f(sum)) * kLn2;
    }
}

template <int KC, int VC, bool E4>
int launch_generic(const ChunkArgs &a) {
    const int group = a.num_q_heads / a.cache.num_kv_heads;
    const int parts = (group + kHeads - 1) / kHeads;
    const size_t smem = sizeof(float) * kWarps * kHeads * (a.cache.head_dim_v + 2);
    auto kernel = chunk_generic_kernel<KC, VC, E4>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) !=
            cudaSuccess)
        return PKV_ERR_CUDA;
    return launch_pdl(kernel, dim3(a.num_tokens, a.cache.num_kv_heads * parts), dim3(kWarps * 32),
                      smem, a.stream, a);
}

template <bool E4>
int launch_dims(const ChunkArgs &a) {
    const int kc = (a.cache.head_dim_k / 8 + 31) / 32, vc = (a.cache.head_dim_v / 8 + 31) / 32;
    if (kc <= 1 && vc <= 1) return launch_generic<1, 1, E4>(a);
    if (kc <= 3 && vc <= 2) return launch_generic<3, 2, E4>(a);
    return launch_generic<4, 4, E4>(a);
}

}  // namespace

int launch_chunk_generic(const ChunkArgs &a) { return launch_dims<false>(a); }
int launch_chunk_generic_e4m3(const ChunkArgs &a) { return launch_dims<true>(a); }

}  // namespace pkv
