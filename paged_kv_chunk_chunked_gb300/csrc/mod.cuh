// Modified scores, shared by the attention kernels: a tanh cap, a bias that
// falls with distance, and a range of visible keys per query.
//
//   s_ij = q_i . k_j / sqrt(d);  s <- c tanh(s / c);  s <- s - slope_h |i - j|;
//   j visible to i iff k_begin[i] <= j < k_end[i].
// The cap's derivative is 1 - tanh^2. A row that sees nothing has O = 0,
// LSE = -inf and no gradient.
#pragma once

#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {

// The keys [lo, hi) visible to query row i of the chunk; (0, 0) if none.
// Positions fit 32 bits: a pool holds fewer than 2^31 rows.
__device__ __forceinline__ int2 row_range(const ModArgs& m, int64_t q_start, int64_t i) {
    const int64_t lo = m.k_begin ? max64(m.k_begin[i], 0) : 0;
    const int64_t hi = m.k_end ? min64(m.k_end[i], m.n_keys) : q_start + i + 1;
    return hi > lo ? make_int2((int)lo, (int)hi) : make_int2(0, 0);
}

// Bounds over a tile of query rows: keys outside [lo, hi) are visible to none
// of them (lo = hi = 0: no row sees anything), keys in [full_lo, full_hi) to all.
struct TileRange {
    int lo, hi, full_lo, full_hi;
};

// Of rows [row0, row0 + ROWS) of the chunk, those past n_q left out; by one
// warp, the same result in every lane.
template <int ROWS>
__device__ __forceinline__ TileRange tile_range(const ModArgs& m, int64_t q_start, int64_t row0, int64_t n_q, int lane) {
    TileRange t{0x7fffffff, 0, 0, 0x7fffffff};
    if (!m.k_begin && !m.k_end) {
        t.lo = 0;
        t.hi = (int)(q_start + min64(row0 + ROWS, n_q));
        t.full_hi = (int)(q_start + row0 + 1);
        return t;
    }
#pragma unroll
    for (int k = 0; k < ROWS / 32; ++k) {
        const int64_t i = row0 + k * 32 + lane;
        if (i >= n_q) continue;
        const int2 r = row_range(m, q_start, i);
        if (r.y > 0) {
            t.lo = min(t.lo, r.x);
            t.hi = max(t.hi, r.y);
        }
        t.full_lo = max(t.full_lo, r.x);
        t.full_hi = min(t.full_hi, r.y);
    }
    t.lo = __reduce_min_sync(0xffffffffu, t.lo);
    t.hi = __reduce_max_sync(0xffffffffu, t.hi);
    t.full_lo = __reduce_max_sync(0xffffffffu, t.full_lo);
    t.full_hi = __reduce_min_sync(0xffffffffu, t.full_hi);
    if (t.hi == 0) t.lo = 0;
    return t;
}

// tanh(u) for |u| <= 1: u times a polynomial in u^2 fitted to tanh(u) / u by
// iteratively reweighted least squares (a minimax fit), within 1.2e-7 in fp32.
__device__ __forceinline__ float tanh_small(float u) {
    const float w = u * u;
    float p = 0.0010410224786028266f;
    p = fmaf(p, w, -0.006203378550708294f);
    p = fmaf(p, w, 0.020289979875087738f);
    p = fmaf(p, w, -0.05345702916383743f);
    p = fmaf(p, w, 0.13325203955173492f);
    p = fmaf(p, w, -0.33332839608192444f);
    p = fmaf(p, w, 0.9999999403953552f);
    return u * p;
}

// tanh(u) for any u: 1 - 2 / (1 + e^(2u)), absolute error below 3e-7 (the
// division is exact to an ulp; u = +-inf gives +-1).
__device__ __forceinline__ float tanh_any(float u) {
    return 1.f - __fdividef(2.f, 1.f + fast_exp2(u * (2.f * kLog2e)));
}

}  // namespace pkv
