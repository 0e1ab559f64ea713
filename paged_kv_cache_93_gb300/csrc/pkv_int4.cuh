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
// bf16 because the values are: from bf16 rows it is exact.  A scale rounded to bf16 is
// off by 2^-9 at most, 0.03 of a step at the row's far end.  A spread below 15 * 2^-126
// is stored as none (scale 0, codes 0).  A row with an element that is infinite or NaN,
// or whose spread is no binary32, is stored as scale = offset = NaN and reads as NaN.
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

// `low` and `high` of the row; a row that holds an infinite or NaN element comes with
// low = -inf, high = +inf.
__device__ __forceinline__ Int4Scale int4_scale(float low, float high) {
    Int4Scale r;
    const uint32_t o = f32_to_bf16_bits(low);
    r.offset = __uint_as_float(o << 16);
    const float range = fmaxf(__fsub_rn(high, r.offset), 0.f);
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

// Eight elements as codes, the first in the low bits.  Adding 2^23 rounds to the nearest
// whole number (ties to even) and leaves it in the low bits of the sum.
__device__ __forceinline__ uint32_t int4_codes8(const float (&x)[8], const Int4Scale &r) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float v = __fmul_rn(__fsub_rn(x[i], r.offset), r.inverse);
        // (a NaN element's row has NaN parameters; fmaxf makes its code 0)
        const float c = __fadd_rn(fminf(fmaxf(v, 0.f), 15.f), 8388608.f);
        w = (w << 4) | (__float_as_uint(c) & 15u);
    }
    return w;
}

// Takes eight elements into a row's running smallest and largest; `odd` becomes NaN when
// one of them is infinite or NaN, and stays 0 otherwise.
__device__ __forceinline__ void int4_extent8(const float (&x)[8], float &low, float &high,
                                             float &odd) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        low = fminf(low, x[i]);
        high = fmaxf(high, x[i]);
        odd = fmaf(x[i], 0.f, odd);
    }
}

// The same over the `lanes` (a power of two) neighbouring lanes that hold a row's
// elements; the lanes of `mask` call it together.
__device__ __forceinline__ Int4Scale int4_row_scale(float low, float high, float odd,
                                                    int lanes, uint32_t mask) {
    if (odd != 0.f) {
        low = -INFINITY;
        high = INFINITY;
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(mask, low, o));
        high = fmaxf(high, __shfl_xor_sync(mask, high, o));
    }
    return int4_scale(low, high);
}

}  // namespace pkv
