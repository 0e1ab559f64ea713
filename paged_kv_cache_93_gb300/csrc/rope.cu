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
// signed number of 2^-32 turns, are rounded to binary32 (2^-26 turns) for
// sincospif.
//
// Bound: memory.  Every q, k and v element is read once and written once, as
// 16-byte vectors; cosines and sines (rotary_dim / 2 of them against (Hq + Hkv) *
// head_dim elements) are computed once for all of a token's heads, or for a part of
// them: in a warp's registers for the common heads, in shared memory for the others.
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
    uint32_t tok_magic;                  // of a token's units, where tokens are grouped
    int32_t group, parts;                // tokens of a work item; items of a token
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

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
// 8 elements to `at`..`at`+7 (at a multiple of 8) as bf16, fp32 or codes; bf16 ones that
// are only copied go as the bytes they came in, so that a NaN keeps its bits.
__device__ __forceinline__ void store8_raw(void *p, int64_t at, const uint4 &x) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) = x;
}
__device__ __forceinline__ void store8_bf16(void *p, int64_t at, const float (&f)[8]) {
    store8_raw(p, at, pack8(f));
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
            // elements outside the rotary part
            auto copy8 = [&](int e) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + e);
                if (is_q ? a.q_fp32 != 0 : E4) {
                    float x[8];
                    unpack8(v, x);
                    store8(e, x);
                } else {
                    store8_raw(is_q ? a.q_out : a.k_pool, dst + e, v);
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
                    copy8(e);
                }
            } else if constexpr (VEC) {
                const int e = c * 8;
                if (e >= a.off && e < a.off + a.rot) {
                    float x[8];
                    unpack8(*reinterpret_cast<const uint4 *>(src + e), x);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 r = tab[((e - a.off) >> 1) + i];
                        const float p = x[2 * i], s = x[2 * i + 1];
                        x[2 * i] = p * r.x - s * r.y;
                        x[2 * i + 1] = s * r.x + p * r.y;
                    }
                    store8(e, x);
                } else if (!(is_q && a.in_place)) {
                    copy8(e);
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
                    if (is_q ? a.q_fp32 != 0 : E4)
                        store1(e, __uint_as_float(uint32_t(src[e]) << 16));
                    else
                        static_cast<uint16_t *>(is_q ? a.q_out : a.k_pool)[dst + e] = src[e];
                }
            }
        }
        buf ^= 1;      // the other table: this one may still be read by slower warps
    }
}

// The form for rows that split into units of 16 elements (head dims, rotary_dim and
// rotary_offset multiples of 16).  A unit is two 16-byte vectors: of the two halves
// of the rotary part (half layout), or neighbours.  A thread keeps one unit
// position and walks rows (a token's query heads, key heads, value heads, then the
// next token's), so that only the row is left to be worked out for each unit; the
// instructions, not the bytes, are what a simpler mapping was bound by.  A CTA takes
// `group` tokens, or 1 / parts of one with many heads, at a time; kAhead units of
// the next rows are loaded while the last ones are turned and stored (1,024 latent
// tokens of 128 heads of 576: 60.5 us, 5.0 TB/s).
constexpr int kAhead = 2;
constexpr int kWideCtas = 3;             // per SM
constexpr int kItemUnits = 2048;         // units of a work item, about
constexpr int kTable = 1024;             // entries of a table of cosines and sines

template <bool INTER, bool E4>
__global__ void __launch_bounds__(kThreads, kWideCtas)
rope_append_wide_kernel(const RopeArgs a) {
    __shared__ __align__(16) float2 cs[2][kTable];   // (cos, sin) * amplitude
    __shared__ uint64_t step[kMaxPairs];
    __shared__ int64_t s_slot[2][8];             // slot of a token's rows, or -1: not stored
    __shared__ int32_t s_live[2][8];
    const int npairs = a.rot >> 1;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < npairs; i += kThreads) step[i] = turn_step(a.inv_freq[i]);
    __syncthreads();
    // this thread's unit of a row, and the row it takes first
    const int r0 = fast_div(threadIdx.x, a.q_magic, a.q_units), c = threadIdx.x - r0 * a.q_units;
    const int rows_pass = kThreads / a.q_units;      // rows a pass of the CTA covers
    const bool works = r0 < rows_pass;
    const int rows_qk = a.hq + a.hkv, rows_tok = rows_qk + (a.dv ? a.hkv : 0);
    bool turned;
    int ea, eb;
    if constexpr (INTER) {
        ea = 16 * c;
        eb = ea + 8;
        turned = ea >= a.off && ea < a.off + a.rot;
    } else {
        turned = c < (a.rot >> 4);
        ea = turned ? a.off + 8 * c : 16 * (c - (a.rot >> 4));
        if (!turned && ea >= a.off) ea += a.rot;
        eb = turned ? ea + (a.rot >> 1) : ea + 8;
    }
    // A unit's eight pairs are four 16-byte entries of the table, kept so that
    // neighbouring units' entries are neighbours (no bank conflicts): entry i of
    // unit u at i * (rotary units) + u.
    const int nr = a.rot >> 4, unit = INTER ? c - (a.off >> 4) : c;
    const int64_t groups = (a.num_tokens + a.group - 1) / a.group;
    int buf = 0;
    for (int64_t w = blockIdx.x; w < groups * a.parts; w += gridDim.x) {
        const int64_t grp = a.parts > 1 ? w / a.parts : w;
        const int part = a.parts > 1 ? int(w - grp * a.parts) : 0;
        const int64_t t0 = grp * a.group;
        const int ntok = int(a.num_tokens - t0 < a.group ? a.num_tokens - t0 : a.group);
        const int per = (rows_tok + a.parts - 1) / a.parts;
        const int begin = part * per;
        const int end = a.parts > 1 ? min(rows_tok, begin + per) : ntok * rows_tok;
        auto load = [&](int row, uint4 &va, uint4 &vb) {
            if (!works || row >= end) return;
            const int tk = a.group > 1 ? fast_div(row, a.tok_magic, rows_tok) : 0;
            row -= tk * rows_tok;
            const int64_t t = t0 + tk;
            const uint16_t *src;
            int e0 = ea, e1 = eb;
            if (row < a.hq) {
                src = a.q + (t * a.hq + row) * a.dk;
            } else if (row < rows_qk) {
                src = a.k_new + (t * a.hkv + row - a.hq) * a.dk;
            } else {
                if (16 * c >= a.dv) return;
                src = a.v_new + (t * a.hkv + row - rows_qk) * a.dv;
                e0 = 16 * c;
                e1 = e0 + 8;
            }
            va = *reinterpret_cast<const uint4 *>(src + e0);
            vb = *reinterpret_cast<const uint4 *>(src + e1);
        };
        auto turn_unit = [&](int tk, float (&x)[8], float (&y)[8]) {
            const float4 *r =
                reinterpret_cast<const float4 *>(cs[buf] + tk * npairs) + unit;
            if constexpr (INTER) {
                auto turn = [](float (&v)[8], int i, const float4 &q) {
                    float p = v[4 * i], s = v[4 * i + 1];
                    v[4 * i] = p * q.x - s * q.y;
                    v[4 * i + 1] = s * q.x + p * q.y;
                    p = v[4 * i + 2], s = v[4 * i + 3];
                    v[4 * i + 2] = p * q.z - s * q.w;
                    v[4 * i + 3] = s * q.z + p * q.w;
                };
                turn(x, 0, r[0]);
                turn(x, 1, r[nr]);
                turn(y, 0, r[2 * nr]);
                turn(y, 1, r[3 * nr]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 q = r[i * nr];
                    float p = x[2 * i], s = y[2 * i];
                    x[2 * i] = p * q.x - s * q.y;
                    y[2 * i] = s * q.x + p * q.y;
                    p = x[2 * i + 1], s = y[2 * i + 1];
                    x[2 * i + 1] = p * q.z - s * q.w;
                    y[2 * i + 1] = s * q.z + p * q.w;
                }
            }
        };
        auto finish = [&](int row, uint4 va, uint4 vb) {
            if (!works || row >= end) return;
            const int tk = a.group > 1 ? fast_div(row, a.tok_magic, rows_tok) : 0;
            row -= tk * rows_tok;
            const int64_t slot = s_slot[buf][tk];
            const bool is_q = row < a.hq;
            if (is_q ? !s_live[buf][tk] || (a.in_place && !turned) : slot < 0) return;
            const bool is_k = !is_q && row < rows_qk;
            if (!is_q && !is_k && 16 * c >= a.dv) return;
            const int g = is_k ? row - a.hq : row - rows_qk, d = is_k ? a.dk : a.dv;
            const int e0 = is_q || is_k ? ea : 16 * c, e1 = is_q || is_k ? eb : 16 * c + 8;
            // s_slot holds the row of KV head 0
            const int64_t dst = is_q ? ((t0 + tk) * a.hq + row) * a.dk
                                     : (slot + int64_t(g) * a.block_size) * d;
            if (is_q ? !a.q_fp32 : !E4) {
                // to bf16: copied elements as they came
                if (turned && (is_q || is_k)) {
                    float x[8], y[8];
                    unpack8(va, x);
                    unpack8(vb, y);
                    turn_unit(tk, x, y);
                    va = pack8(x);
                    vb = pack8(y);
                }
                void *to = is_q ? a.q_out : is_k ? a.k_pool : a.v_pool;
                store8_raw(to, dst + e0, va);
                store8_raw(to, dst + e1, vb);
                return;
            }
            float x[8], y[8];
            unpack8(va, x);
            unpack8(vb, y);
            if (turned && (is_q || is_k)) turn_unit(tk, x, y);
            if (is_q) {
                store8_f32(a.q_out, dst + e0, x);
                store8_f32(a.q_out, dst + e1, y);
            } else {
                const float s = (is_k ? a.k_scale : a.v_scale)[g];
                store8_e4m3(is_k ? a.k_pool : a.v_pool, dst + e0, x, s);
                store8_e4m3(is_k ? a.k_pool : a.v_pool, dst + e1, y, s);
            }
        };
        uint4 va[2][kAhead], vb[2][kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            load(begin + k * rows_pass + r0, va[0][k], vb[0][k]);
        // the tokens' slots and angles, while the first units come in
        if (threadIdx.x < ntok) {
            const int64_t slot = a.slots[t0 + threadIdx.x];
            const int64_t pos = a.positions[t0 + threadIdx.x];
            const bool stored = pos >= 0 && slot >= 0 && slot < a.num_slots;
            if (pos >= 0 && slot >= a.num_slots) raise_status(a.status, PKV_DEV_SLOT);
            const int64_t block = stored ? slot / a.block_size : 0;
            s_slot[buf][threadIdx.x] =
                stored ? block * a.hkv * a.block_size + (slot - block * a.block_size) : -1;
            s_live[buf][threadIdx.x] = pos >= 0;
        }
        for (int i = threadIdx.x; i < ntok * npairs; i += kThreads) {
            const int tk = a.group > 1 ? i / npairs : 0, pr = i - tk * npairs;
            const uint64_t turn = step[pr] * uint64_t(a.positions[t0 + tk]);
            // signed 2^-32 turns; sincospif takes half turns
            const float x = float(int32_t(turn >> 32)) * 4.656612873077393e-10f;
            float s, co;
            sincospif(x, &s, &co);
            const int entry = ((pr >> 1) & 3) * nr + (pr >> 3);
            cs[buf][tk * npairs + 2 * entry + (pr & 1)] =
                make_float2(co * a.amplitude, s * a.amplitude);
        }
        __syncthreads();
        const int pass = rows_pass * kAhead;
        for (int row = begin + r0; row < end + r0; row += 2 * pass) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int here = row + half * pass;
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    load(here + pass + k * rows_pass, va[half ^ 1][k], vb[half ^ 1][k]);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    finish(here + k * rows_pass, va[half][k], vb[half][k]);
            }
        }
        buf ^= 1;      // the other table: this one may still be read by slower warps
    }
}

// The form for the common heads: head_dim_k = head_dim_v (or values inside the keys)
// of 64, 128, 256 or 512 and at most 128 rotary elements.  A warp takes a token, or one
// of its `parts`: 32 / U rows at a time (U = head_dim / 16 units a row), each lane the
// same unit of every row, with the cosines and sines of its eight pairs in
// registers -- two pairs a lane are computed, then handed round by shuffles -- so
// that rows need neither table nor barrier, and the rows kWarpAhead passes on are
// on their way (8,191 tokens of 32 + 8 heads of 128: 36.9 us, 5.5 TB/s, against 37.7
// for 4 ahead on two CTAs an SM; 2,500 tokens of 64 + 8 heads into an FP8 cache:
// 24.8 us against 35.7).
constexpr int kWarpAhead = 2;
constexpr int kWarpCtas = 3;             // per SM

template <bool INTER, bool E4>
__global__ void __launch_bounds__(kThreads, kWarpCtas)
rope_append_warp_kernel(const RopeArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int U = a.q_units, shift = 31 - __clz(U), rpp = 32 >> shift;
    const int c = lane & (U - 1), r0 = lane >> shift, nr = a.rot >> 4, npairs = a.rot >> 1;
    bool turned;
    int ea, eb, unit;
    if constexpr (INTER) {
        unit = c - (a.off >> 4);
        turned = unit >= 0 && unit < nr;
        ea = 16 * c;
        eb = ea + 8;
    } else {
        unit = c;
        turned = c < nr;
        ea = turned ? a.off + 8 * c : 16 * (c - nr);
        if (!turned && ea >= a.off) ea += a.rot;
        eb = turned ? ea + (a.rot >> 1) : ea + 8;
    }
    // this lane's pairs: lane and lane + 32
    uint64_t step[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        step[i] = lane + 32 * i < npairs ? turn_step(a.inv_freq[lane + 32 * i]) : 0;
    const int pq = (a.hq + rpp - 1) >> (5 - shift), pk = (a.hkv + rpp - 1) >> (5 - shift);
    const int passes = pq + pk + (a.dv ? pk : 0), per = (passes + a.parts - 1) / a.parts;
    const int64_t items = a.num_tokens * a.parts;
    const int warps = gridDim.x * (kThreads / 32);
    for (int64_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); w < items; w += warps) {
        const int64_t t = a.parts > 1 ? w / a.parts : w;
        const int begin = a.parts > 1 ? int(w - t * a.parts) * per : 0;
        const int end = min(passes, begin + per);
        const int64_t pos = a.positions[t], slot = a.slots[t];
        uint4 va[kWarpAhead], vb[kWarpAhead];
        // pass p: rows of queries, keys, then values
        auto load = [&](int p, uint4 &x, uint4 &y) {
            if (p >= end) return;
            const uint16_t *src;
            int row, heads, e0 = ea, e1 = eb;
            if (p < pq) {
                row = (p << (5 - shift)) + r0;
                heads = a.hq;
                src = a.q;
            } else {
                const bool is_k = p < pq + pk;
                row = ((p - pq - (is_k ? 0 : pk)) << (5 - shift)) + r0;
                heads = a.hkv;
                src = is_k ? a.k_new : a.v_new;
                if (!is_k) {
                    e0 = 16 * c;
                    e1 = e0 + 8;
                }
            }
            if (row >= heads) return;
            src += (t * heads + row) * a.dk;
            x = *reinterpret_cast<const uint4 *>(src + e0);
            y = *reinterpret_cast<const uint4 *>(src + e1);
        };
        if (pos < 0) continue;                       // padding (the whole warp)
#pragma unroll
        for (int k = 0; k < kWarpAhead; ++k) load(begin + k, va[k], vb[k]);
        // ---- the angles
        float co[8], si[8];
        {
            float c2[2], s2[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint64_t turn = step[i] * uint64_t(pos);
                // signed 2^-32 turns; sincospif takes half turns
                sincospif(float(int32_t(turn >> 32)) * 4.656612873077393e-10f, &s2[i], &c2[i]);
                c2[i] *= a.amplitude;
                s2[i] *= a.amplitude;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pr = (8 * unit + j) & 63;
                const float cl = __shfl_sync(0xffffffffu, c2[0], pr & 31);
                const float ch = __shfl_sync(0xffffffffu, c2[1], pr & 31);
                const float sl = __shfl_sync(0xffffffffu, s2[0], pr & 31);
                const float sh = __shfl_sync(0xffffffffu, s2[1], pr & 31);
                co[j] = pr < 32 ? cl : ch;
                si[j] = pr < 32 ? sl : sh;
            }
        }
        if (slot >= a.num_slots && lane == 0 && begin == 0) raise_status(a.status, PKV_DEV_SLOT);
        const bool stored = slot >= 0 && slot < a.num_slots;
        const int64_t block = stored ? slot / a.block_size : 0;
        const int64_t row0 = block * a.hkv * a.block_size + (stored ? slot - block * a.block_size : 0);
        auto turn = [&](float (&x)[8], float (&y)[8]) {
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = x[2 * i], s0 = x[2 * i + 1];
                    x[2 * i] = p0 * co[i] - s0 * si[i];
                    x[2 * i + 1] = s0 * co[i] + p0 * si[i];
                    const float p1 = y[2 * i], s1 = y[2 * i + 1];
                    y[2 * i] = p1 * co[4 + i] - s1 * si[4 + i];
                    y[2 * i + 1] = s1 * co[4 + i] + p1 * si[4 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p0 = x[i], s0 = y[i];
                    x[i] = p0 * co[i] - s0 * si[i];
                    y[i] = s0 * co[i] + p0 * si[i];
                }
            }
        };
        auto finish = [&](int p, uint4 va, uint4 vb) {
            if (p >= end) return;
            const bool is_q = p < pq, is_k = !is_q && p < pq + pk;
            const int row = ((p - (is_q ? 0 : is_k ? pq : pq + pk)) << (5 - shift)) + r0;
            if (row >= (is_q ? a.hq : a.hkv)) return;
            if (is_q ? a.in_place && !turned : !stored) return;
            const int64_t dst =
                (is_q ? t * a.hq + row : row0 + int64_t(row) * a.block_size) * a.dk;
            if (is_q ? !a.q_fp32 : !E4) {
                // to bf16: copied elements as they came
                if (turned && (is_q || is_k)) {
                    float x[8], y[8];
                    unpack8(va, x);
                    unpack8(vb, y);
                    turn(x, y);
                    va = pack8(x);
                    vb = pack8(y);
                }
                void *to = is_q ? a.q_out : is_k ? a.k_pool : a.v_pool;
                store8_raw(to, dst + (is_q || is_k ? ea : 16 * c), va);
                store8_raw(to, dst + (is_q || is_k ? eb : 16 * c + 8), vb);
                return;
            }
            float x[8], y[8];
            unpack8(va, x);
            unpack8(vb, y);
            if (turned && (is_q || is_k)) turn(x, y);
            if (is_q) {
                store8_f32(a.q_out, dst + ea, x);
                store8_f32(a.q_out, dst + eb, y);
            } else {
                const float s = (is_k ? a.k_scale : a.v_scale)[row];
                store8_e4m3(is_k ? a.k_pool : a.v_pool, dst + (is_k ? ea : 16 * c), x, s);
                store8_e4m3(is_k ? a.k_pool : a.v_pool, dst + (is_k ? eb : 16 * c + 8), y, s);
            }
        };
        for (int p = begin; p < end; p += kWarpAhead)
#pragma unroll
            for (int k = 0; k < kWarpAhead; ++k) {
                const uint4 x = va[k], y = vb[k];
                load(p + kWarpAhead + k, va[k], vb[k]);
                finish(p + k, x, y);
            }
    }
}

uint32_t magic_of(int n) { return n > 1 ? uint32_t(((uint64_t(1) << 32) + n - 1) / n) : 0; }

template <bool E4>
int launch_warp(RopeArgs &a, bool interleaved, cudaStream_t stream) {
    // Parts of a token: the fewest rounds of warps x (passes of a part + 2 for its
    // angles), so that few tokens spread over the device and the last round of
    // many is not mostly empty.
    constexpr int per_cta = kThreads / 32;
    const int64_t warps = int64_t(sm_count()) * kWarpCtas * per_cta;
    const int rpp = 32 / a.q_units;
    const int passes = (a.hq + rpp - 1) / rpp + (a.dv ? 2 : 1) * ((a.hkv + rpp - 1) / rpp);
    a.parts = 1;
    int64_t least = INT64_MAX;
    for (int parts = 1; parts <= std::min(passes, 32); ++parts) {
        const int64_t cost = (a.num_tokens * parts + warps - 1) / warps *
                             ((passes + parts - 1) / parts + 2);
        if (cost < least) {
            least = cost;
            a.parts = parts;
        }
    }
    const int64_t items = a.num_tokens * a.parts;
    const dim3 grid(unsigned(std::min<int64_t>((items + per_cta - 1) / per_cta,
                                               int64_t(sm_count()) * kWarpCtas)));
    return launch_pdl(interleaved ? rope_append_warp_kernel<true, E4>
                                  : rope_append_warp_kernel<false, E4>,
                      grid, dim3(kThreads), 0, stream, a);
}

template <bool E4>
int launch(RopeArgs &a, bool interleaved, cudaStream_t stream) {
    const int64_t units16 =
        (int64_t(a.hq) + a.hkv) * (a.dk / 16) + int64_t(a.hkv) * (a.dv / 16);
    const int units = a.dk / 16;
    if (a.dk % 64 == 0 && (units & (units - 1)) == 0 && units <= 32 &&
        (a.dv == 0 || a.dv == a.dk) && a.rot % 16 == 0 && a.off % 16 == 0 && a.rot <= 128) {
        a.q_units = units;
        return launch_warp<E4>(a, interleaved, stream);
    }
    if (a.dk % 16 == 0 && a.dv % 16 == 0 && a.dv <= a.dk && a.rot % 16 == 0 && a.off % 16 == 0) {
        a.q_units = a.dk / 16;
        a.q_magic = magic_of(a.q_units);
        a.tok_magic = magic_of(a.hq + a.hkv + (a.dv ? a.hkv : 0));
        // few tokens: one each, over as many CTAs as there are; more: groups of
        // about kItemUnits units, as many tokens as the table holds at most
        const int64_t ctas = int64_t(sm_count()) * kWideCtas;
        int64_t group = std::min<int64_t>(
            {int64_t(8), kItemUnits / units16, int64_t(kTable / (a.rot / 2)), a.num_tokens / ctas});
        a.group = int32_t(std::max<int64_t>(1, group));
        a.parts = a.group > 1 ? 1 : int32_t((units16 + kItemUnits - 1) / kItemUnits);
        const int64_t items = (a.num_tokens + a.group - 1) / a.group * a.parts;
        const dim3 grid(unsigned(std::min(items, ctas)));
        return launch_pdl(interleaved ? rope_append_wide_kernel<true, E4>
                                      : rope_append_wide_kernel<false, E4>,
                          grid, dim3(kThreads), 0, stream, a);
    }
    const bool vec = interleaved ? (a.rot % 8 == 0 && a.off % 8 == 0)
                                 : (a.rot % 16 == 0 && a.off % 8 == 0);
    a.q_units = !vec          ? a.rot / 2 + (a.dk - a.rot)
                : interleaved ? a.dk / 8
                              : a.rot / 16 + (a.dk - a.rot) / 8;
    a.v_units = a.dv / 8;
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
