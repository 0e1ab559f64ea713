// rope.cu -- rotary positions of the new tokens' queries and keys, fused with
// the scatter of keys and values into the paged cache.
//
// Pair i of a head's rotary part, (x1, x2), is turned by the angle
// position * inv_freq[i]:
//     (x1, x2) -> amplitude * (x1 cos - x2 sin, x2 cos + x1 sin)
// with (x1, x2) = elements (i, i + R/2) of the rotary part (half layout) or
// (2i, 2i + 1) (interleaved), R = rotary_dim.
//
// The angle.  A far position times a frequency is many turns, of which only
// the fraction matters: in binary32 position 200,000 would leave an angle
// error of about 1e-2.  So the frequency is held as a 64-bit fixed-point
// fraction of a turn, F = frac(inv_freq / 2 pi) * 2^64, and position * F in
// wrapping 64-bit integer arithmetic IS the fraction of a turn, off by at most
// position * 2^-53 turns (F comes from a binary64).  Its upper 32 bits, as a
// signed number of 2^-32 turns, go to sincospif.
//
// Bound: memory.  Every q, k and v element is read once and written once, as
// 16-byte vectors; the tokens' cosines and sines are computed once per token
// into shared memory (rotary_dim / 2 of them against (Hq + Hkv) * head_dim
// elements) and shared by all heads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv.h"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;           // head dims up to 1024

struct RopeArgs {
    const uint16_t *q, *k_new, *v_new;   // bf16
    const int64_t *positions, *slots;
    const double *inv_freq;
    const float *k_scale, *v_scale;      // E4M3 pools
    void *k_pool, *v_pool, *q_out;
    uint32_t *status;
    int64_t num_tokens, num_slots;
    int32_t hq, hkv, dk, dv;             // dv 0: values inside the keys
    int32_t block_size;
    int32_t rot, off;                    // rotary_dim, rotary_offset
    int32_t q_units, v_units;            // work units of a q/k row and of a v row
    uint32_t q_magic, v_magic;           // ceil(2^32 / units): index -> row
    float amplitude;
    int32_t q_fp32, in_place;
};

// x / n for x * n < 2^32, by multiplication with magic = ceil(2^32 / n).
__device__ __forceinline__ int fast_div(int x, uint32_t magic, int n) {
    return n == 1 ? x : int(__umulhi(uint32_t(x), magic));
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    f[0] = bf16_lo_to_f32(u.x); f[1] = bf16_hi_to_f32(u.x);
    f[2] = bf16_lo_to_f32(u.y); f[3] = bf16_hi_to_f32(u.y);
    f[4] = bf16_lo_to_f32(u.z); f[5] = bf16_hi_to_f32(u.z);
    f[6] = bf16_lo_to_f32(u.w); f[7] = bf16_hi_to_f32(u.w);
}

// 8 values to elements `at`..`at`+7 (at a multiple of 8) as bf16, fp32 or codes.
__device__ __forceinline__ void store8_bf16(void *p, int64_t at, const float (&f)[8]) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8_f32(void *p, int64_t at, const float (&f)[8]) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
}
// The code nearest to x / scale (the quotient rounded to binary32), as
// pkv_kv_append_e4m3 stores it; here x is the rotated key before any rounding
// to bf16.
__device__ __forceinline__ void store8_e4m3(void *p, int64_t at, const float (&f)[8], float s) {
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        c[i] = e4m3x2_from_f32(__fdiv_rn(f[4 * i], s), __fdiv_rn(f[4 * i + 1], s)) |
               e4m3x2_from_f32(__fdiv_rn(f[4 * i + 2], s), __fdiv_rn(f[4 * i + 3], s)) << 16;
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p) + at) = make_uint2(c[0], c[1]);
}

// Fraction-of-a-turn increment per position of a frequency in radians.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
    const double turns = inv_freq * 0.15915494309189535;      // 1 / (2 pi)
    return __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
}

// VEC: rotary_dim and rotary_offset let whole 16-byte vectors rotate (half
// layout: both multiples of 16 and 8; interleaved: multiples of 8).  Otherwise
// a unit is a single pair, or a single element outside the rotary part.
template <bool INTER, bool E4, bool VEC>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(const RopeArgs a) {
    __shared__ float2 cs[2][kMaxPairs];          // (cos, sin) * amplitude, by token parity
    const int npairs = a.rot >> 1;
    pdl_wait();
    pdl_launch_dependents();
    // this thread's frequencies (kMaxPairs / kThreads at most)
    uint64_t step[kMaxPairs / kThreads];
#pragma unroll
    for (int i = 0; i < kMaxPairs / kThreads; ++i) {
        const int pr = threadIdx.x + i * kThreads;
        step[i] = pr < npairs ? turn_step(a.inv_freq[pr]) : 0;
    }
    const int rows_qk = a.hq + a.hkv;
    const int n_qk = rows_qk * a.q_units, n_all = n_qk + a.hkv * a.v_units;
    int buf = 0;
    for (int64_t t = blockIdx.x; t < a.num_tokens; t += gridDim.x) {
        const int64_t pos = a.positions[t];
        if (pos < 0) continue;                   // padding (uniform in the CTA)
        const int64_t slot = a.slots[t];
        float2 *tab = cs[buf];
#pragma unroll
        for (int i = 0; i < kMaxPairs / kThreads; ++i) {
            const int pr = threadIdx.x + i * kThreads;
            if (pr < npairs) {
                const uint64_t turn = step[i] * uint64_t(pos);
                // signed 2^-32 turns; sincospif takes half turns
                const float x = float(int32_t(turn >> 32)) * 4.656612873077393e-10f;
                float s, c;
                sincospif(x, &s, &c);
                tab[pr] = make_float2(c * a.amplitude, s * a.amplitude);
            }
        }
        const bool stored = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && threadIdx.x == 0) raise_status(a.status, PKV_DEV_SLOT);
        const int64_t block = stored ? slot / a.block_size : 0;
        const int64_t off_tok = stored ? slot - block * a.block_size : 0;
        __syncthreads();
        for (int u = threadIdx.x; u < n_all; u += kThreads) {
            if (u >= n_qk) {
                // ---- a value vector: copied (or quantised) into its pool
                const int w = u - n_qk;
                const int g = fast_div(w, a.v_magic, a.v_units), c = (w - g * a.v_units) * 8;
                if (!stored) continue;
                const uint4 x = *reinterpret_cast<const uint4 *>(
                    a.v_new + (t * a.hkv + g) * a.dv + c);
                const int64_t dst =
                    ((block * a.hkv + g) * a.block_size + off_tok) * a.dv + c;
                if constexpr (E4) {
                    float f[8];
                    unpack8(x, f);
                    store8_e4m3(a.v_pool, dst, f, a.v_scale[g]);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.v_pool) + dst) = x;
                }
                continue;
            }
            const int row = fast_div(u, a.q_magic, a.q_units), c = u - row * a.q_units;
            const bool is_q = row < a.hq;
            const int g = row - a.hq;
            if (!is_q && !stored) continue;
            const uint16_t *src = is_q ? a.q + (t * a.hq + row) * a.dk
                                       : a.k_new + (t * a.hkv + g) * a.dk;
            const int64_t dst =
                is_q ? (t * a.hq + row) * a.dk
                     : ((block * a.hkv + g) * a.block_size + off_tok) * a.dk;
            auto store8 = [&](int e, const float (&f)[8]) {
                if (is_q) {
                    if (a.q_fp32) store8_f32(a.q_out, dst + e, f);
                    else store8_bf16(a.q_out, dst + e, f);
                } else if constexpr (E4) {
                    store8_e4m3(a.k_pool, dst + e, f, a.k_scale[g]);
                } else {
                    store8_bf16(a.k_pool, dst + e, f);
                }
            };
            auto store1 = [&](int e, float x) {
                if (is_q) {
                    if (a.q_fp32) static_cast<float *>(a.q_out)[dst + e] = x;
                    else static_cast<uint16_t *>(a.q_out)[dst + e] = uint16_t(f32_to_bf16_bits(x));
                } else if constexpr (E4) {
                    static_cast<uint8_t *>(a.k_pool)[dst + e] =
                        uint8_t(e4m3x2_from_f32(__fdiv_rn(x, a.k_scale[g]), 0.f));
                } else {
                    static_cast<uint16_t *>(a.k_pool)[dst + e] = uint16_t(f32_to_bf16_bits(x));
                }
            };
            if constexpr (VEC && !INTER) {
                // units: rot / 16 vector pairs, then the vectors outside
                const int nr = a.rot >> 4;
                if (c < nr) {
                    const int e1 = a.off + c * 8, e2 = e1 + (a.rot >> 1);
                    float x[8], y[8];
                    const uint4 vx = *reinterpret_cast<const uint4 *>(src + e1);
                    const uint4 vy = *reinterpret_cast<const uint4 *>(src + e2);
                    unpack8(vx, x);
                    unpack8(vy, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 r = tab[c * 8 + i];
                        const float p = x[i], s = y[i];
                        x[i] = p * r.x - s * r.y;
                        y[i] = s * r.x + p * r.y;
                    }
                    store8(e1, x);
                    store8(e2, y);
                } else if (!(is_q && a.in_place)) {
                    int e = (c - nr) * 8;
                    if (e >= a.off) e += a.rot;
                    float x[8];
                    unpack8(*reinterpret_cast<const uint4 *>(src + e), x);
                    store8(e, x);
                }
            } else if constexpr (VEC) {
                const int e = c * 8;
                const bool turned = e >= a.off && e < a.off + a.rot;
                if (turned || !(is_q && a.in_place)) {
                    float x[8];
                    unpack8(*reinterpret_cast<const uint4 *>(src + e), x);
                    if (turned) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 r = tab[((e - a.off) >> 1) + i];
                            const float p = x[2 * i], s = x[2 * i + 1];
                            x[2 * i] = p * r.x - s * r.y;
                            x[2 * i + 1] = s * r.x + p * r.y;
                        }
                    }
                    store8(e, x);
                }
            } else {
                // units: rot / 2 pairs, then the elements outside
                if (c < npairs) {
                    const int e1 = a.off + (INTER ? 2 * c : c), e2 = e1 + (INTER ? 1 : npairs);
                    const float2 r = tab[c];
                    const float p = __uint_as_float(uint32_t(src[e1]) << 16);
                    const float s = __uint_as_float(uint32_t(src[e2]) << 16);
                    store1(e1, p * r.x - s * r.y);
                    store1(e2, s * r.x + p * r.y);
                } else if (!(is_q && a.in_place)) {
                    int e = c - npairs;
                    if (e >= a.off) e += a.rot;
                    store1(e, __uint_as_float(uint32_t(src[e]) << 16));
                }
            }
        }
        buf ^= 1;      // the other table: this one may still be read by slower warps
    }
}

uint32_t magic_of(int n) { return n > 1 ? uint32_t(((uint64_t(1) << 32) + n - 1) / n) : 0; }

template <bool E4>
int launch(RopeArgs &a, bool interleaved, cudaStream_t stream) {
    const bool vec = interleaved ? (a.rot % 8 == 0 && a.off % 8 == 0)
                                 : (a.rot % 16 == 0 && a.off % 8 == 0);
    a.q_units = !vec          ? a.rot / 2 + (a.dk - a.rot)
                : interleaved ? a.dk / 8
                              : a.rot / 16 + (a.dk - a.rot) / 8;
    a.v_units = std::max(1, a.dv / 8);
    if (a.dv == 0) a.v_units = 0;
    a.q_magic = magic_of(a.q_units);
    a.v_magic = magic_of(std::max(1, a.v_units));
    const dim3 grid(unsigned(std::min<int64_t>(a.num_tokens, int64_t(sm_count()) * 8)));
    auto kernel = interleaved
                      ? (vec ? rope_append_kernel<true, E4, true> : rope_append_kernel<true, E4, false>)
                      : (vec ? rope_append_kernel<false, E4, true>
                             : rope_append_kernel<false, E4, false>);
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, a);
}

// The host checks both entry points share; fills everything but the pools'
// scales.  *done: nothing to launch.
int prepare(RopeArgs &a, bool e4, const pkv_cache_desc *c, const void *q, int32_t hq,
            const void *k_new, const void *v_new, const int64_t *positions, const int64_t *slots,
            int64_t num_tokens, const double *inv_freq, int32_t rotary_dim, int32_t rotary_offset,
            float amplitude, int32_t flags, void *k_pool, void *v_pool, void *q_out, bool *done) {
    *done = false;
    if (!c || num_tokens < 0 || hq <= 0 || (flags & ~(PKV_ROPE_INTERLEAVED | PKV_ROPE_Q_FP32)) ||
        !std::isfinite(amplitude))
        return PKV_ERR_INVALID_ARG;
    if (c->num_blocks <= 0 || c->block_size < 1 || c->block_size > 256 || c->num_kv_heads <= 0 ||
        c->head_dim_k <= 0 || c->head_dim_v <= 0 || c->head_dim_k % 8 != 0 ||
        c->head_dim_v % 8 != 0 || c->head_dim_k > 1024 || c->head_dim_v > 1024)
        return PKV_ERR_INVALID_ARG;
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_offset < 0 ||
        rotary_offset > c->head_dim_k - rotary_dim)
        return PKV_ERR_SHAPE;
    // rows x units of a token stay within the index division's range
    if (int64_t(hq) + c->num_kv_heads > 4096) return PKV_ERR_SHAPE;
    if (num_tokens == 0) {
        *done = true;
        return PKV_OK;
    }
    if (!q || !q_out || !k_new || !k_pool || !positions || !slots || !inv_freq ||
        !v_pool != !v_new)
        return PKV_ERR_INVALID_ARG;
    if (!v_pool && (e4 || c->head_dim_v > c->head_dim_k))
        return e4 ? PKV_ERR_INVALID_ARG : PKV_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k_new) || (v_new && !aligned16(v_new)))
        return PKV_ERR_ALIGNMENT;
    const uintptr_t pool_mask = e4 ? 7 : 15;
    if ((reinterpret_cast<uintptr_t>(k_pool) & pool_mask) ||
        (reinterpret_cast<uintptr_t>(v_pool) & pool_mask))
        return PKV_ERR_ALIGNMENT;
    const bool fp32 = (flags & PKV_ROPE_Q_FP32) != 0;
    if (fp32 && q_out == q) return PKV_ERR_INVALID_ARG;      // wider than its input
    a.status = status_word();
    if (!a.status) return PKV_ERR_CUDA;
    a.q = static_cast<const uint16_t *>(q);
    a.k_new = static_cast<const uint16_t *>(k_new);
    a.v_new = static_cast<const uint16_t *>(v_new);
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.q_out = q_out;
    a.num_tokens = num_tokens;
    a.num_slots = int64_t(c->num_blocks) * c->block_size;
    a.hq = hq;
    a.hkv = c->num_kv_heads;
    a.dk = c->head_dim_k;
    a.dv = v_pool ? c->head_dim_v : 0;
    a.block_size = c->block_size;
    a.rot = rotary_dim;
    a.off = rotary_offset;
    a.amplitude = amplitude;
    a.q_fp32 = fp32;
    a.in_place = q_out == q;
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_rope_frequencies(int32_t rotary_dim, double theta, double factor,
                                    double original_len, double low_turns, double high_turns,
                                    double *inv_freq) {
    if (rotary_dim < 2 || rotary_dim % 2 != 0 || !(theta > 0) || !std::isfinite(theta) ||
        !(factor >= 1) || !std::isfinite(factor) || !inv_freq)
        return PKV_ERR_INVALID_ARG;
    const bool by_parts = original_len != 0;
    if (by_parts && (!(original_len > 0) || !std::isfinite(original_len) || !(low_turns > 0) ||
                     !(high_turns > low_turns) || !std::isfinite(high_turns)))
        return PKV_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / rotary_dim);
        double keep = 0.0;          // share of the unscaled frequency
        if (by_parts) {
            const double turns = original_len * f / kTwoPi;
            keep = std::min(1.0, std::max(0.0, (turns - low_turns) / (high_turns - low_turns)));
        }
        inv_freq[i] = keep * f + (1.0 - keep) * (f / factor);
    }
    return PKV_OK;
}

extern "C" int pkv_rope_append(const pkv_cache_desc *cache, void *k_pool, void *v_pool,
                               const void *q, int32_t num_q_heads, const void *k_new,
                               const void *v_new, const int64_t *positions,
                               const int64_t *slot_mapping, int64_t num_tokens,
                               const double *inv_freq, int32_t rotary_dim, int32_t rotary_offset,
                               float amplitude, int32_t flags, void *q_out, pkv_stream_t stream) {
    RopeArgs a = {};
    bool done;
    const int rc = prepare(a, false, cache, q, num_q_heads, k_new, v_new, positions, slot_mapping,
                           num_tokens, inv_freq, rotary_dim, rotary_offset, amplitude, flags,
                           k_pool, v_pool, q_out, &done);
    if (rc != PKV_OK || done) return rc;
    return launch<false>(a, flags & PKV_ROPE_INTERLEAVED, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int pkv_rope_append_e4m3(const pkv_cache_desc *cache, void *k_pool, void *v_pool,
                                    const void *q, int32_t num_q_heads, const void *k_new,
                                    const void *v_new, const float *k_scale,
                                    const float *v_scale, const int64_t *positions,
                                    const int64_t *slot_mapping, int64_t num_tokens,
                                    const double *inv_freq, int32_t rotary_dim,
                                    int32_t rotary_offset, float amplitude, int32_t flags,
                                    void *q_out, pkv_stream_t stream) {
    RopeArgs a = {};
    bool done;
    const int rc = prepare(a, true, cache, q, num_q_heads, k_new, v_new, positions, slot_mapping,
                           num_tokens, inv_freq, rotary_dim, rotary_offset, amplitude, flags,
                           k_pool, v_pool, q_out, &done);
    if (rc != PKV_OK || done) return rc;
    if (!k_scale || !v_scale) return PKV_ERR_INVALID_ARG;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    return launch<true>(a, flags & PKV_ROPE_INTERLEAVED, reinterpret_cast<cudaStream_t>(stream));
}
