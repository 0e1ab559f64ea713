// chunk_merge_units.h -- how the warps of chunk attention's merge walk its work:
// first `units` of each of `entries` (a split item of one KV head), unit-major, so that
// the units past a short item's rows end up in other warps than its rows; then
// `rest` further pieces.  entries * units may pass 2^31 (2^29 query rows, up to 32
// units), so a warp's place is kept as unit and entry and stepped by quotient and
// remainder of its stride: 32-bit arithmetic, and no division in the loop.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__
#else
#define PKV_HOST_DEVICE
#endif

namespace pkv {

struct MergeWalk {
    int32_t entries, units, rest;
    int32_t unit, entry, unit_step, entry_step;

    // Warp `first` of `stride`.
    PKV_HOST_DEVICE MergeWalk(int32_t first, int32_t stride, int32_t entries_, int32_t units_,
                              int32_t rest_)
        : entries(entries_), units(entries_ > 0 ? units_ : 0), rest(rest_) {
        const int32_t n = entries > 0 ? entries : INT32_MAX;
        unit = first / n;
        entry = first - unit * n;
        unit_step = stride / n;
        entry_step = stride - unit_step * n;
    }
    // The piece is an entry's (unit, entry)
    PKV_HOST_DEVICE bool in_entries() const { return unit < units; }
    // or, when it is not, the rest's with this number (rest or more: no more work).
    PKV_HOST_DEVICE int32_t piece() const { return (unit - units) * entries + entry; }
    PKV_HOST_DEVICE bool done() const { return !in_entries() && piece() >= rest; }
    PKV_HOST_DEVICE void next() {
        unit += unit_step;
        entry += entry_step;
        if (entries > 0 && entry >= entries) {
            entry -= entries;
            ++unit;
        }
    }
};

}  // namespace pkv
