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

// The polynomials of tanh (see tanh_long2): ranges, and the short one's coefficients.
constexpr float kTanhShort = 0.4f, kTanhLong = 0.75f;
constexpr float kTanhA[4] = {0.9999998807907104f, -0.33331361413002014f, 0.13270977139472961f, -0.04755360260605812f};

// Sets the cap c (0: none) for head dimension d.
inline void set_cap(ModArgs* m, float c, int d) {
    m->cap = c;
    m->k = m->c2 = m->a0 = m->a1 = m->a2 = m->a3 = m->neg_c2sq = 0.f;
    if (!(c > 0.f)) return;
    const double k = 1.0 / sqrt((double)d) / c, c2 = (double)c * 1.4426950408889634;
    const double u2 = k * k;
    m->k = (float)k;
    m->c2 = (float)c2;
    m->a0 = (float)(kTanhA[0] * c2 * k);
    m->a1 = (float)(kTanhA[1] * c2 * k * u2);
    m->a2 = (float)(kTanhA[2] * c2 * k * u2 * u2);
    m->a3 = (float)(kTanhA[3] * c2 * k * u2 * u2 * u2);
    m->neg_c2sq = (float)(-1.0 / (c2 * c2));
}

// The keys [lo, hi) visible to query row i of the chunk; (0, 0) if none.
// Positions fit 32 bits: a pool holds fewer than 2^31 rows.
__device__ __forceinline__ int2 row_range(const int64_t* k_begin, const int64_t* k_end, int64_t n_keys, int64_t q_start,
                                          int64_t i) {
    const int64_t lo = k_begin ? max64(k_begin[i], 0) : 0;
    const int64_t hi = k_end ? min64(k_end[i], n_keys) : q_start + i + 1;
    return hi > lo ? make_int2((int)lo, (int)hi) : make_int2(0, 0);
}
__device__ __forceinline__ int2 row_range(const ModArgs& m, int64_t q_start, int64_t i) {
    return row_range(m.k_begin, m.k_end, m.n_keys, q_start, i);
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

// Whether a row of [row0, row1) of the chunk sees a key of [k0, k1); by one warp, the
// same result in every lane. For pages whose block-table entry is unusable: the hull of
// a tile's ranges may hold pages that no row sees, and those need no slot. (Out of
// line: inside, it cost the kernels spilled registers.)
static __device__ __noinline__ bool rows_see(const int64_t* k_begin, const int64_t* k_end, int64_t n_keys, int64_t q_start,
                                             int64_t row0, int64_t row1, int k0, int k1) {
    bool any = false;
    for (int64_t i = row0 + threadIdx.x % 32; i < row1; i += 32) {
        const int2 r = row_range(k_begin, k_end, n_keys, q_start, i);
        any |= r.x < k1 && r.y > k0;
    }
    return __any_sync(0xffffffffu, any);
}
template <int ROWS>
__device__ __forceinline__ bool tile_sees(const ModArgs& m, int64_t q_start, int64_t row0, int64_t n_q, int k0, int k1) {
    return rows_see(m.k_begin, m.k_end, m.n_keys, q_start, row0, min64(row0 + ROWS, n_q), k0, k1);
}

// Pairs of floats: one instruction for two elements (sm_100 on). Sums, products
// and fmas are the single ones', element by element.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// tanh(u) = u p(u^2), p a polynomial fitted to tanh(u) / u by iteratively
// reweighted least squares (a minimax fit). The fp32 pipe bounds the capped
// kernels, so the degree follows the largest |u| of a warp's tile rows: capped
// logits are mostly far below their cap.
//   |u| <= 0.4:  4 terms, relative error 9.8e-8, with the cap's constants folded
//                into the coefficients (ModArgs): 5 operations from the raw logit
//                to the score in log2 units;
//   |u| <= 0.75: 6 terms, relative error 2.9e-8, 9 operations;
//   beyond:      through the exponential, two special-function operations; its
//                absolute error, 3e-7 of the cap, is ten times fp32's own for caps of
//                1e3 and more whose logits come near them.
// (The forward's masked tiles, and its tiles with both cap and bias, go straight from
// the short form to the exponential.)
// 28 heads, d 128, 4096 queries on 16384 keys: without a cap the forward takes
// 562 us and the backward 1843 us; with the short form 774 and 2280 us, through the
// exponential 1193 and 3060 us.
__device__ __forceinline__ f32x2 tanh_long2(f32x2 u) {
    const f32x2 w = mul2(u, u);
    f32x2 p = pack2(-0.004716257099062204f, -0.004716257099062204f);
    p = fma2(p, w, pack2(0.01958290860056877f, 0.01958290860056877f));
    p = fma2(p, w, pack2(-0.05334442853927612f, -0.05334442853927612f));
    p = fma2(p, w, pack2(0.1332540661096573f, 0.1332540661096573f));
    p = fma2(p, w, pack2(-0.33332958817481995f, -0.33332958817481995f));
    p = fma2(p, w, pack2(1.f, 1.f));
    return mul2(u, p);
}

// tanh(u) for any u: 1 - 2 / (1 + e^(2u)), absolute error below 3e-7;
// u = +-inf gives +-1.
__device__ __forceinline__ float tanh_any(float u) {
    return 1.f - __fdividef(2.f, 1.f + fast_exp2(u * (2.f * kLog2e)));
}

// Largest of three, and of three magnitudes (one instruction, sm_100 on).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int N> __device__ __forceinline__ float abs_max(const uint32_t (&x)[N]) {
    float b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N; c += 2)
        b[(c >> 1) & 3] = max3_abs(b[(c >> 1) & 3], __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
    return max3(fmaxf(b[0], b[1]), b[2], b[3]);
}

template <int N> __device__ __forceinline__ f32x2 pair_at(const uint32_t (&x)[N], int c) {
    return pack2(__uint_as_float(x[c]), __uint_as_float(x[c + 1]));
}
template <int N> __device__ __forceinline__ void put_pair(uint32_t (&x)[N], int c, f32x2 v) {
    float a, b;
    unpack2(v, a, b);
    x[c] = __float_as_uint(a);
    x[c + 1] = __float_as_uint(b);
}
template <int N, typename F> __device__ __forceinline__ void each_pair(const uint32_t (&x)[N], F&& use) {
#pragma unroll
    for (int c = 0; c < N; c += 2) use(c, pair_at(x, c));
}

// The cap over a row of a tile: use(c, y) gets the scores of raw logits x[c],
// x[c + 1] in log2 units. `top`: the largest |x| of the warp's rows, which picks
// the form for the whole warp.
template <int N, typename F>
__device__ __forceinline__ void cap_short(const uint32_t (&x)[N], const ModArgs& m, F&& use) {
    const f32x2 a0 = pack2(m.a0, m.a0), a1 = pack2(m.a1, m.a1), a2 = pack2(m.a2, m.a2), a3 = pack2(m.a3, m.a3);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const f32x2 v = pair_at(x, c), w = mul2(v, v);
        use(c, mul2(v, fma2(fma2(fma2(a3, w, a2), w, a1), w, a0)));
    }
}
template <int N, typename F>
__device__ __forceinline__ void cap_long(const uint32_t (&x)[N], const ModArgs& m, F&& use) {
    const f32x2 k = pack2(m.k, m.k), c2 = pack2(m.c2, m.c2);
#pragma unroll
    for (int c = 0; c < N; c += 2) use(c, mul2(tanh_long2(mul2(pair_at(x, c), k)), c2));
}
template <int N, typename F>
__device__ __forceinline__ void cap_any(const uint32_t (&x)[N], const ModArgs& m, F&& use) {
#pragma unroll
    for (int c = 0; c < N; c += 2)
        use(c, pack2(m.c2 * tanh_any(__uint_as_float(x[c]) * m.k), m.c2 * tanh_any(__uint_as_float(x[c + 1]) * m.k)));
}
template <int N, typename F>
__device__ __forceinline__ void cap_pairs(const uint32_t (&x)[N], const ModArgs& m, float top, F&& use) {
    if (top * m.k <= kTanhShort) {
        cap_short(x, m, use);
    } else if (top * m.k <= kTanhLong) {
        cap_long(x, m, use);
    } else {
        cap_any(x, m, use);
    }
}
// Every lane's largest over the warp (of values >= 0; their bits order as integers).
__device__ __forceinline__ float warp_top(float x) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

// The distance bias over a row of a tile: use(c, y) gets x * pre + bias of
// elements c, c + 1, where element c lies at distance d0 + dir * c from the row's
// own position. Where the whole tile lies on one side (`side`, the sign of the
// distance) the bias is linear in c, one operation to form it; tiles across the
// diagonal (side 0) need the magnitude.
template <int N, typename F>
__device__ __forceinline__ void bias_pairs(const uint32_t (&x)[N], float pre, float slope2, float d0, float dir, int side,
                                           F&& use) {
    const f32x2 pp = pack2(pre, pre);
    if (side != 0) {
        const float base = -slope2 * (float)side * d0, step = -slope2 * (float)side * dir;
#pragma unroll
        for (int c = 0; c < N; c += 2)
            use(c, fma2(pair_at(x, c), pp, pack2(fmaf(step, (float)c, base), fmaf(step, (float)(c + 1), base))));
    } else {
#pragma unroll
        for (int c = 0; c < N; c += 2)
            use(c, fma2(pair_at(x, c), pp, pack2(-slope2 * fabsf(fmaf(dir, (float)c, d0)),
                                                 -slope2 * fabsf(fmaf(dir, (float)(c + 1), d0)))));
    }
}

}  // namespace pkv
