// What the cache and the attention kernels share: which sequence a workgroup works for, and the
// checked reading of the batch's device values.
#pragma once

#include "device.h"
#include "kv_internal.h"

namespace bgf {

// cu_tokens[i] held to [0, T]: whatever the array holds, no row outside the batch is reached.
__device__ __forceinline__ int cu_at(const KvView& c, int i) { return min(max(c.cu[i], 0), c.T); }

// A launch covers a ragged batch with slots: sequence s owns the slots base(s) .. base(s + 1) - 1,
// base(s) = cu[s] * mul / div + per * s. That many suffice for ceil(n * mul / div) row tiles
// (per = 1), or for the pages that n tokens touch wherever they begin (mul = 1, div = page, per = 2),
// and the grid is exact to `per` slots a sequence without the host knowing any length.
// Returns the sequence of `slot` (-1: none) and its first slot. All lanes of the wave take part: each
// step tests 64 places, so up to 64 sequences take one round trip to memory and 4096 take two.
__device__ __forceinline__ int slot_base(const KvView& c, int s, int mul, int div, int per) {
    return (int)((unsigned)cu_at(c, s) * (unsigned)mul / (unsigned)div) + per * s;
}
__device__ __forceinline__ int find_sequence(const KvView& c, int slot, int mul, int div, int per, int* first) {
    const int lane = __lane_id();
    int lo = 0, hi = c.S;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) >> 6;
        const int i = lo + lane * step;
        const bool in = i < hi && slot_base(c, i, mul, div, per) <= slot;
        const int n = __popcll(__ballot(in));
        if (n == 0) return -1;
        lo += (n - 1) * step;
        hi = min(lo + step, hi);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    *first = __builtin_amdgcn_readfirstlane(slot_base(c, lo, mul, div, per));
    return *first <= slot ? lo : -1;
}

// page idx of a sequence's table row, or -1 where the table has none or holds no page number
__device__ __forceinline__ int page_at(const KvView& c, int s, int idx) {
    if (idx < 0 || idx >= c.W) return -1;
    const int p = c.table[(int64_t)s * c.table_ld + idx];
    return (p >= 0 && (int64_t)p < c.pages) ? p : -1;
}

// 2^(code - 127) of an E8M0 code as fp32 (code 0 -> 0: see the callers)
__device__ __forceinline__ float e8m0_value(uint32_t code) { return __uint_as_float(code << 23); }

}  // namespace bgf
