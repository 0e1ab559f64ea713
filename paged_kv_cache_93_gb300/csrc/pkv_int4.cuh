// pkv_int4.cuh -- the 4-bit cache's rows, shared by the kernels that write them.
//
// A row (one token, one KV head) of D elements is D / 2 bytes of codes, element 2i in
// the low and 2i + 1 in the high half of byte i, and a bf16 pair (scale, offset):
// element d reads back as scale * code[d] + offset.  With `low` and `high` the row's
// smallest and largest element:
//     offset = bf16(low),  scale = bf16((high - offset) * fl(1/15)),
//     code = the whole number nearest to (x - offset) * fl(1 / scale), ties to even,
//            held within 0..15
// each operation rounded to binary32.  The offset is the row's own smallest value and
// not a whole number of steps, so that rows far from zero keep their spread, and in
// bf16 because the values are: from bf16 rows it is exact.  A scale rounded to bf16 (8
// significant bits) is off by 2^-8 of itself at most, 0.06 of a step at the row's far end.
// A spread below 15 * 2^-126 is stored as none (scale 0, codes 0).  A row with an element
// that is infinite or NaN, or whose spread is no binary32, is stored as scale = offset =
// NaN and reads as NaN.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {

constexpr float kFloatMax = 3.402823466e38f;
constexpr uint32_t kInt4NanParams = 0x7fc07fc0u;

struct Int4Scale {
    float offset, inverse;
    uint32_t params;               // bf16 pair: scale in bits 0-15, offset in 16-31
};

// min and max that give NaN where an operand is NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
    float x;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float x;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t x;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(a), "r"(b));
    return x;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t x;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(a), "r"(b));
    return x;
}

// `low` and `high` of the row, NaN if an element is.
__device__ __forceinline__ Int4Scale int4_scale(float low, float high) {
    Int4Scale r;
    const uint32_t o = f32_to_bf16_bits(low);
    r.offset = __uint_as_float(o << 16);
    float range = __fsub_rn(high, r.offset);
    if (range < 0.f) range = 0.f;
    if (!(range <= kFloatMax)) {
        r.offset = r.inverse = 0.f;
        r.params = kInt4NanParams;
        return r;
    }
    uint32_t s = f32_to_bf16_bits(__fmul_rn(range, 1.0f / 15.0f));
    if (s < 0x80u) s = 0;          // below 2^-126
    r.inverse = s ? __frcp_rn(__uint_as_float(s << 16)) : 0.f;
    r.params = s | (o << 16);
    return r;
}

// Two binary32 operations at a time, each rounded as by itself.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
    return x;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t x;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
    return x;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t x;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
    return x;
}

// Eight elements as codes, the first in the low bits.  Adding 2^23 rounds to the nearest
// whole number (ties to even) and leaves it in the low bits of the sum, whose other bits
// are 0x4b000000; a word is made by multiplying by 16 and adding, and what those bits add
// up to is taken off at the end.  (A code cannot pass 15: the scale is short of
// range / 15 by 2^-8 of it at most, so that the largest quotient, 15.06 with binary32's
// own roundings, is below 15.5.  In a row of NaN parameters max makes codes 0.)
__device__ __forceinline__ uint32_t int4_codes8(const float (&x)[8], const Int4Scale &r) {
    const uint64_t less = pair_of(-r.offset, -r.offset), by = pair_of(r.inverse, r.inverse);
    const uint64_t magic = pair_of(8388608.f, 8388608.f);
    uint32_t w = 0;
#pragma unroll
    for (int i = 6; i >= 0; i -= 2) {
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;"
            : "=f"(lo), "=f"(hi) : "l"(mul2(add2(pair_of(x[i], x[i + 1]), less), by)));
        uint32_t a, b;
        asm("mov.b64 {%0, %1}, %2;"
            : "=r"(a), "=r"(b) : "l"(add2(pair_of(fmaxf(lo, 0.f), fmaxf(hi, 0.f)), magic)));
        w = (w * 16u + b) * 16u + a;
    }
    return w - 0x4b000000u * 0x11111111u;
}

// Takes eight elements into a row's running smallest and largest.
__device__ __forceinline__ void int4_extent8(const float (&x)[8], float &low, float &high) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        low = min_nan(low, x[i]);
        high = max_nan(high, x[i]);
    }
}

// The same over the `lanes` (a power of two) neighbouring lanes that hold a row's
// elements; the lanes of `mask` call it together.
__device__ __forceinline__ Int4Scale int4_row_scale(float low, float high, int lanes,
                                                    uint32_t mask) {
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        low = min_nan(low, __shfl_xor_sync(mask, low, o));
        high = max_nan(high, __shfl_xor_sync(mask, high, o));
    }
    return int4_scale(low, high);
}

}  // namespace pkv
