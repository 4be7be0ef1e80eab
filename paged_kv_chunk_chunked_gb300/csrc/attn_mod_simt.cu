// CUDA-core attention with modified scores (mod.cuh), forward and backward,
// fp32 arithmetic: fp32 pools, and bf16 pools whose pages the tensor-core
// kernels do not take.
//
// The rows of a tile are (query, head) pairs of one KV group: row r of KV head
// kvh is query r / g, head kvh * g + r % g. Short chunks fill their tiles this
// way, and a key tile is read once for the group's heads. Keys are fetched row
// by row through the block table, so pages of any size and ranges that start
// inside a page need no care.
//
//   fwd     CTA per (16 rows, KV head, share of the keys): online softmax over
//           tiles of 64 keys, O in registers. Thread (rg, kg): rows rg, rg + 8,
//           keys kg + 16 j; its O columns are float4s kg * 4 + 64 j.
//   dQ      CTA per (16 rows, KV head), four groups of 128 threads on tiles of 32
//           keys in turn; P from LSE, dS through shared memory.
//   dK/dV   CTA per (16 keys, KV head), four groups on the row tiles that see them
//           in turn; one plain addition per gradient element (a key has one owner).
// The backward's groups add their parts in a fixed order at the end: the sizes
// this path is for make few CTAs, and one group's tiles one after another took
// three times as long (2 heads, 64 queries on 256 keys: dQ 28 us, dK/dV 35 us).
// Rows of K in shared memory are D + 4 floats apart: the 8 threads of a
// 128-byte phase read 8 consecutive rows' 16 bytes from 8 different bank groups.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mod.cuh"

namespace pkv {
namespace {

constexpr int BM = 16, BN = 64, NT = 128;

// Exact scores of these kernels: natural units, tanhf.
__device__ __forceinline__ void mod_score(const ModArgs& m, float slope, float scale, float dot, int dist, float& y, float& f) {
    y = dot * scale;
    f = 1.f;
    if (m.cap > 0.f) {
        const float t = tanhf(y / m.cap);
        y = m.cap * t;
        f = fmaf(-t, t, 1.f);
    }
    y = fmaf(-slope, (float)abs(dist), y);
}

// Rows of one tile: `n` of them from row `r0` of KV head kvh on; with a
// selection a tile lies inside one query page.
struct RowTile {
    int64_t r0;
    int n;
    int qp;
};
__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, int64_t t) {
    const int g = a.Hq / a.Hkv;
    RowTile x;
    if (!a.sel) {
        x.r0 = t * BM;
        x.n = (int)min64(BM, a.n_q * g - x.r0);
        x.qp = 0;
        return x;
    }
    const int64_t per = ((int64_t)a.P * g + BM - 1) / BM;       // tiles of a query page
    x.qp = (int)(t / per);
    const int64_t first = (int64_t)x.qp * a.P * g, off = (t - x.qp * per) * BM;
    x.r0 = first + off;
    x.n = (int)max64(0, min64(BM, min64((int64_t)a.P * g - off, a.n_q * g - x.r0)));
    return x;
}
int64_t row_tiles(const AttnArgs& a) {
    const int64_t g = a.Hq / a.Hkv;
    if (!a.sel) return (a.n_q * g + BM - 1) / BM;
    return (a.n_q + a.P - 1) / a.P * ((a.P * g + BM - 1) / BM);
}

// Offset of row r of KV head kvh in a [n_q, Hq, D] tensor, and its head.
__device__ __forceinline__ size_t row_offset(const AttnArgs& a, int64_t r, int kvh, int D) {
    const int g = a.Hq / a.Hkv;
    return ((size_t)(r / g) * a.Hq + kvh * g + r % g) * D;
}

template <typename T, int D>
__device__ __forceinline__ void load_row_tile(float (*dst)[D + 4], const void* src, const AttnArgs& a, const RowTile& t,
                                              int kvh, int tid, int threads = NT) {
    constexpr int EPV = 16 / (int)sizeof(T), VPR = D / EPV;
    for (int i = tid; i < BM * VPR; i += threads) {
        const int r = i / VPR, v = i % VPR;
        float f[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) f[e] = 0.f;
        if (r < t.n)
            widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(src) + row_offset(a, t.r0 + r, kvh, D)) + v), f);
#pragma unroll
        for (int e = 0; e < EPV; e += 4)
            *reinterpret_cast<float4*>(&dst[r][v * EPV + e]) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
}

// Keys first, first + step, .. below end, some of them without a usable page: an error
// where a row of the tile sees one.
__device__ __noinline__ void bad_keys(const int32_t* bt, int64_t num_phys, int P, int64_t first, int64_t end, int step,
                                      const int2* range, int* err) {
    for (int64_t key = first; key < end; key += step) {
        const int32_t pp = bt[key / P];
        if (pp >= 0 && pp < num_phys) continue;
        bool seen = !range;
        for (int u = 0; range && u < BM; ++u) seen |= (int)key >= range[u].x && (int)key < range[u].y;
        if (seen) report_error(err, kErrBadPage);
    }
}

// Keys k0 .. k0 + n - 1 (n <= N; rows behind read as zero) of K and V. Keys whose
// block-table entry is out of range read as zero, which is an error where a row of
// the tile sees the key (`range`: the rows' keys; null: some row does).
template <typename T, int D, int N>
__device__ __forceinline__ void load_key_tile(float (*Ks)[D + 4], float (*Vs)[D + 4], const AttnArgs& a, int64_t k0, int n,
                                              int kvh, const int2* range, int tid, int threads = NT) {
    constexpr int EPV = 16 / (int)sizeof(T), VPR = D / EPV;
    bool bad = false;
    for (int i = tid; i < N * VPR; i += threads) {
        const int r = i / VPR, v = i % VPR;
        float fk[EPV], fv[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) fk[e] = fv[e] = 0.f;
        if (r < n) {
            const int64_t key = k0 + r, lp = key / a.P;
            const int32_t pp = a.bt[lp];
            if (pp < 0 || pp >= a.num_phys) {
                bad = true;
            } else {
                const size_t off = (((size_t)pp * a.Hkv + kvh) * a.P + (size_t)(key - lp * a.P)) * D;
                widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.kpool) + off) + v), fk);
                widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.vpool) + off) + v), fv);
            }
        }
#pragma unroll
        for (int e = 0; e < EPV; e += 4) {
            *reinterpret_cast<float4*>(&Ks[r][v * EPV + e]) = make_float4(fk[e], fk[e + 1], fk[e + 2], fk[e + 3]);
            *reinterpret_cast<float4*>(&Vs[r][v * EPV + e]) = make_float4(fv[e], fv[e + 1], fv[e + 2], fv[e + 3]);
        }
    }
    // (Of the threads that share a row, the first.)
    if (bad && tid % VPR == 0) bad_keys(a.bt, a.num_phys, a.P, k0 + tid / VPR, k0 + n, threads / VPR, range, a.err);
}

__device__ __forceinline__ float dot4(const float4& x, const float4& y, float acc) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc))));
}

// Smallest and one past the largest key that the tile's rows see.
__device__ __forceinline__ int2 tile_keys(const int2 (&range)[BM]) {
    int lo = 0x7fffffff, hi = 0;
#pragma unroll
    for (int r = 0; r < BM; ++r)
        if (range[r].y > 0) {
            lo = min(lo, range[r].x);
            hi = max(hi, range[r].y);
        }
    return hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// Calls f(k0, n) for the key tiles of up to N keys that a row tile sees: of
// the share blockIdx.z of its range (dense), or of its query page's list.
template <int N, typename F>
__device__ __forceinline__ void for_key_tiles(const AttnArgs& a, const RowTile& t, int kvh, int2 keys, F&& f) {
    if (!a.sel) {
            const int n = (keys.y - keys.x + N - 1) / N;
        const int t0 = (int)((int64_t)n * blockIdx.z / gridDim.z), t1 = (int)((int64_t)n * (blockIdx.z + 1) / gridDim.z);
        for (int j = t0; j < t1; ++j) f((int64_t)keys.x + j * N, min(N, keys.y - keys.x - j * N));
        return;
    }
    const int32_t* row = a.sel + ((size_t)t.qp * a.Hkv + kvh) * a.kmax;
    for (int i = 0; i < a.kmax; ++i) {
        const int32_t lp = row[i];
        if (lp < 0) break;
        const int p0 = max(lp * a.P, keys.x), p1 = min((lp + 1) * a.P, keys.y);
        for (int k0 = p0; k0 < p1; k0 += N) f((int64_t)k0, min(N, p1 - k0));
    }
}

template <typename T, int D>
struct FwdSmem {
    float Q[BM][D + 4], K[BN][D + 4], V[BN][D + 4], P[BM][BN + 4];
    int2 range[BM];
};

// (4 CTAs per SM: left to itself the compiler takes 80 to 96 registers and spills. bf16,
// 8/2 heads, 512 queries on 2048 keys, pages of 32: d 64 177 -> 171 us.)
template <typename T, int D>
__global__ void __launch_bounds__(NT, 4) fwd_mod_simt(AttnArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& S = *reinterpret_cast<FwdSmem<T, D>*>(smem_raw);
    constexpr int CV = D / 64;                                  // float4 columns per thread
    const int tid = threadIdx.x, rg = tid / 16, kg = tid % 16;
    const int kvh = blockIdx.y, g = a.Hq / a.Hkv;
    const RowTile t = row_tile(a, blockIdx.x);
    if (t.n <= 0) return;
    load_row_tile<T, D>(S.Q, a.q, a, t, kvh, tid);
    if (tid < BM) S.range[tid] = tid < t.n ? row_range(a.m, a.q_start, (t.r0 + tid) / g) : make_int2(0, 0);
    __syncthreads();
    const int2 keys = tile_keys(S.range);
    const float scale = rsqrtf((float)D);
    float m[2], l[2], slope[2];
    int2 rr[2];
    int pos[2];
    float4 o[2][CV];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = rg + 8 * u;
        m[u] = -INFINITY;
        l[u] = 0.f;
        rr[u] = S.range[r];
        const int64_t row = t.r0 + min(r, t.n - 1);
        pos[u] = (int)(a.q_start + row / g);
        slope[u] = a.m.slopes ? a.m.slopes[kvh * g + row % g] : 0.f;
#pragma unroll
        for (int c = 0; c < CV; ++c) o[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for_key_tiles<BN>(a, t, kvh, keys, [&](int64_t k0, int n) {
        __syncthreads();
        load_key_tile<T, D, BN>(S.K, S.V, a, k0, n, kvh, S.range, tid);
        __syncthreads();
        float s[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[u][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qv[2], kv[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) qv[u] = *reinterpret_cast<const float4*>(&S.Q[rg + 8 * u][d]);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(&S.K[kg + 16 * j][d]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[u][j] = dot4(qv[u], kv[j], s[u][j]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = (int)k0 + kg + 16 * j;
                float y, f;
                mod_score(a.m, slope[u], scale, s[u][j], pos[u] - key, y, f);
                s[u][j] = key >= rr[u].x && key < rr[u].y && kg + 16 * j < n ? y : -INFINITY;
                top = fmaxf(top, s[u][j]);
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float m_new = fmaxf(m[u], top);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            const float alpha = expf(m[u] - ref);               // m = -inf: 0, and l = o = 0
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = expf(s[u][j] - ref);
                sum += p;
                S.P[rg + 8 * u][kg + 16 * j] = p;
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[u] = l[u] * alpha + sum;
            m[u] = m_new;
#pragma unroll
            for (int c = 0; c < CV; ++c) {
                o[u][c].x *= alpha; o[u][c].y *= alpha; o[u][c].z *= alpha; o[u][c].w *= alpha;
            }
        }
        __syncwarp();                                           // a row's 16 threads are half a warp
#pragma unroll 2
        for (int k = 0; k < BN; k += 4) {
            float4 p[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) p[u] = *reinterpret_cast<const float4*>(&S.P[rg + 8 * u][k]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < CV; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(&S.V[k + e][kg * 4 + 64 * c]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float w = e == 0 ? p[u].x : e == 1 ? p[u].y : e == 2 ? p[u].z : p[u].w;
                        o[u][c].x = fmaf(w, v.x, o[u][c].x);
                        o[u][c].y = fmaf(w, v.y, o[u][c].y);
                        o[u][c].z = fmaf(w, v.z, o[u][c].z);
                        o[u][c].w = fmaf(w, v.w, o[u][c].w);
                    }
                }
        }
    });
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = rg + 8 * u;
        if (r >= t.n) continue;
        const int64_t row = t.r0 + r;
        const int h = kvh * g + (int)(row % g);
        const size_t hrow = (size_t)h * a.n_q + row / g;
        const float inv = l[u] == 0.f ? 0.f : 1.f / l[u];
        const float lse = l[u] == 0.f ? -INFINITY : m[u] + logf(l[u]);
        if (a.splits > 1) {
            const size_t prow = (size_t)blockIdx.z * a.Hq * a.n_q + hrow;
#pragma unroll
            for (int c = 0; c < CV; ++c)
                *reinterpret_cast<float4*>(a.part + prow * D + kg * 4 + 64 * c) =
                    make_float4(o[u][c].x * inv, o[u][c].y * inv, o[u][c].z * inv, o[u][c].w * inv);
            if (kg == 0) a.part[(size_t)a.splits * a.Hq * a.n_q * D + prow] = lse * kLog2e;
        } else {
            T* dst = static_cast<T*>(a.o) + row_offset(a, row, kvh, D);
#pragma unroll
            for (int c = 0; c < CV; ++c) {
                Elem<T>::store(dst + kg * 4 + 64 * c, o[u][c].x * inv);
                Elem<T>::store(dst + kg * 4 + 64 * c + 1, o[u][c].y * inv);
                Elem<T>::store(dst + kg * 4 + 64 * c + 2, o[u][c].z * inv);
                Elem<T>::store(dst + kg * 4 + 64 * c + 3, o[u][c].w * inv);
            }
            if (kg == 0) a.lse[hrow] = lse;
        }
    }
}

constexpr int kGroups = 4, GT = kGroups * NT;         // the backward's thread groups
constexpr int BNG = 32;                               // keys of a group's tile (dQ)

__device__ __forceinline__ void group_sync(int gi) { asm volatile("bar.sync %0, 128;" :: "r"(1 + gi) : "memory"); }

template <typename T, int D>
struct DqSmem {
    float Q[BM][D + 4], dO[BM][D + 4];
    float K[kGroups][BNG][D + 4], V[kGroups][BNG][D + 4], S[kGroups][BM][BNG + 4];
    int2 range[BM];
};

template <typename T, int D>
__global__ void __launch_bounds__(GT) bwd_dq_mod_simt(AttnArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& S = *reinterpret_cast<DqSmem<T, D>*>(smem_raw);
    constexpr int CV = D / 64;
    const int gi = threadIdx.x / NT, tid = threadIdx.x % NT, rg = tid / 16, kg = tid % 16;
    const int kvh = blockIdx.y, g = a.Hq / a.Hkv;
    const RowTile t = row_tile(a, blockIdx.x);
    if (t.n <= 0) return;
    load_row_tile<T, D>(S.Q, a.q, a, t, kvh, threadIdx.x, GT);
    load_row_tile<T, D>(S.dO, a.dout, a, t, kvh, threadIdx.x, GT);
    if (threadIdx.x < BM)
        S.range[tid] = tid < t.n ? row_range(a.m, a.q_start, (t.r0 + tid) / g) : make_int2(0, 0);
    __syncthreads();
    const int2 keys = tile_keys(S.range);
    const float scale = rsqrtf((float)D);
    float slope[2], lse[2], Dr[2];
    int2 rr[2];
    int pos[2];
    float4 dq[2][CV];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = rg + 8 * u;
        rr[u] = S.range[r];
        const int64_t row = t.r0 + min(r, t.n - 1);
        const int h = kvh * g + (int)(row % g);
        pos[u] = (int)(a.q_start + row / g);
        slope[u] = a.m.slopes ? a.m.slopes[h] : 0.f;
        lse[u] = a.lse_in[(size_t)h * a.n_q + row / g];
        Dr[u] = a.Dbuf[(size_t)h * a.n_q + row / g];
#pragma unroll
        for (int c = 0; c < CV; ++c) dq[u][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int turn = 0;
    for_key_tiles<BNG>(a, t, kvh, keys, [&](int64_t k0, int n) {
        if (turn++ % kGroups != gi) return;
        group_sync(gi);
        load_key_tile<T, D, BNG>(S.K[gi], S.V[gi], a, k0, n, kvh, S.range, tid);
        group_sync(gi);
        float s[2][2], dp[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) s[u][j] = dp[u][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qv[2], ov[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                qv[u] = *reinterpret_cast<const float4*>(&S.Q[rg + 8 * u][d]);
                ov[u] = *reinterpret_cast<const float4*>(&S.dO[rg + 8 * u][d]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 kv = *reinterpret_cast<const float4*>(&S.K[gi][kg + 16 * j][d]);
                const float4 vv = *reinterpret_cast<const float4*>(&S.V[gi][kg + 16 * j][d]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    s[u][j] = dot4(qv[u], kv, s[u][j]);
                    dp[u][j] = dot4(ov[u], vv, dp[u][j]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int key = (int)k0 + kg + 16 * j;
                float y, f;
                mod_score(a.m, slope[u], scale, s[u][j], pos[u] - key, y, f);
                const bool vis = key >= rr[u].x && key < rr[u].y && kg + 16 * j < n;
                S.S[gi][rg + 8 * u][kg + 16 * j] = vis ? expf(y - lse[u]) * (dp[u][j] - Dr[u]) * f : 0.f;
            }
        __syncwarp();                                           // a row's 16 threads are half a warp
#pragma unroll 2
        for (int k = 0; k < BNG; k += 4) {
            float4 w4[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) w4[u] = *reinterpret_cast<const float4*>(&S.S[gi][rg + 8 * u][k]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < CV; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(&S.K[gi][k + e][kg * 4 + 64 * c]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float w = e == 0 ? w4[u].x : e == 1 ? w4[u].y : e == 2 ? w4[u].z : w4[u].w;
                        dq[u][c].x = fmaf(w, v.x, dq[u][c].x);
                        dq[u][c].y = fmaf(w, v.y, dq[u][c].y);
                        dq[u][c].z = fmaf(w, v.z, dq[u][c].z);
                        dq[u][c].w = fmaf(w, v.w, dq[u][c].w);
                    }
                }
        }
    });
    __syncthreads();
    float(*part)[BM][D] = reinterpret_cast<float(*)[BM][D]>(&S.K[0][0][0]);   // [kGroups], over the key tiles
    static_assert(sizeof(S.K) >= kGroups * BM * D * sizeof(float), "the groups' parts fit the key tiles");
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < CV; ++c) *reinterpret_cast<float4*>(&part[gi][rg + 8 * u][kg * 4 + 64 * c]) = dq[u][c];
    __syncthreads();
    for (int i = threadIdx.x; i < t.n * D; i += GT) {
        const int r = i / D, c = i % D;
        Elem<T>::store(static_cast<T*>(a.dq) + row_offset(a, t.r0 + r, kvh, D) + c,
                       ((part[0][r][c] + part[1][r][c]) + (part[2][r][c] + part[3][r][c])) * scale);
    }
}

constexpr int KN = 16;                                          // keys per CTA of the dK/dV kernel

template <typename T, int D>
struct DkvSmem {
    float K[KN][D + 4], V[KN][D + 4];
    float Q[kGroups][BM][D + 4], dO[kGroups][BM][D + 4];
    float P[kGroups][KN][BM + 4], S[kGroups][KN][BM + 4];       // [key][row]
    int2 range[kGroups][BM];
    float lse[kGroups][BM], Dr[kGroups][BM], slope[kGroups][BM];
    int pos[kGroups][BM];
};

// Whether logical page lp is listed for (query page qp, KV head kvh).
__device__ __forceinline__ bool page_listed(const AttnArgs& a, int qp, int kvh, int64_t lp) {
    const int32_t* row = a.sel + ((size_t)qp * a.Hkv + kvh) * a.kmax;
    for (int i = 0; i < a.kmax; ++i) {
        const int32_t x = row[i];
        if (x == lp) return true;
        if (x < 0 || x > lp) return false;                      // ascending, -1 padded
    }
    return false;
}

template <typename T, int D>
__global__ void __launch_bounds__(GT) bwd_dkdv_mod_simt(AttnArgs a, int64_t tiles) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& S = *reinterpret_cast<DkvSmem<T, D>*>(smem_raw);
    constexpr int CV = D / 32;                                  // float4 columns per thread: 8 threads per key
    const int gi = threadIdx.x / NT, tid = threadIdx.x % NT, lane = threadIdx.x % 32;
    const int kvh = blockIdx.y, g = a.Hq / a.Hkv;
    const int64_t k0 = (int64_t)blockIdx.x * KN;                // keys of one page: KN divides the page size
    const int64_t lp = k0 / a.P;
    const int n = (int)min64(KN, a.m.n_keys - k0);
    const int key = tid / 8, sub = tid % 8;                     // score rows sub, sub + 8; columns sub * 4 + 32 c
    const int kpos = (int)k0 + key;
    const float scale = rsqrtf((float)D);
    // Keys that no query sees are not touched (their page need not be staged).
    bool any = false;
    for (int64_t i = threadIdx.x; i < a.n_q && !any; i += GT) {
        const int2 r = row_range(a.m, a.q_start, i);
        any = r.x < (int)k0 + n && r.y > (int)k0 && (!a.sel || page_listed(a, (int)(i / a.P), kvh, lp));
    }
    if (!__syncthreads_or(any)) return;
    load_key_tile<T, D, KN>(S.K, S.V, a, k0, n, kvh, nullptr, threadIdx.x, GT);
    __syncthreads();
    float4 dk[CV], dv[CV];
#pragma unroll
    for (int c = 0; c < CV; ++c) dk[c] = dv[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t ti = gi; ti < tiles; ti += kGroups) {
        const RowTile t = row_tile(a, ti);
        if (t.n <= 0 || (a.sel && !page_listed(a, t.qp, kvh, lp))) continue;   // the same for every thread of the group
        int2 r = make_int2(0, 0);
        if (lane < t.n) r = row_range(a.m, a.q_start, (t.r0 + lane) / g);
        if (!__any_sync(0xffffffffu, r.x < (int)k0 + n && r.y > (int)k0)) continue;   // no row sees these keys
        group_sync(gi);                                         // the group is done with its last tile
        load_row_tile<T, D>(S.Q[gi], a.q, a, t, kvh, tid);
        load_row_tile<T, D>(S.dO[gi], a.dout, a, t, kvh, tid);
        if (tid < BM) {
            const int64_t row = t.r0 + min(tid, t.n - 1);
            const int h = kvh * g + (int)(row % g);
            S.range[gi][tid] = r;
            S.pos[gi][tid] = (int)(a.q_start + row / g);
            S.slope[gi][tid] = a.m.slopes ? a.m.slopes[h] : 0.f;
            S.lse[gi][tid] = a.lse_in[(size_t)h * a.n_q + row / g];
            S.Dr[gi][tid] = a.Dbuf[(size_t)h * a.n_q + row / g];
        }
        group_sync(gi);
        float s[2] = {0.f, 0.f}, dp[2] = {0.f, 0.f};
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            const float4 kv = *reinterpret_cast<const float4*>(&S.K[key][d]);
            const float4 vv = *reinterpret_cast<const float4*>(&S.V[key][d]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                s[u] = dot4(kv, *reinterpret_cast<const float4*>(&S.Q[gi][sub + 8 * u][d]), s[u]);
                dp[u] = dot4(vv, *reinterpret_cast<const float4*>(&S.dO[gi][sub + 8 * u][d]), dp[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = sub + 8 * u;
            float y, f;
            mod_score(a.m, S.slope[gi][i], scale, s[u], S.pos[gi][i] - kpos, y, f);
            const bool vis = key < n && kpos >= S.range[gi][i].x && kpos < S.range[gi][i].y;
            const float p = vis ? expf(y - S.lse[gi][i]) : 0.f;
            S.P[gi][key][i] = p;
            S.S[gi][key][i] = vis ? p * (dp[u] - S.Dr[gi][i]) * f : 0.f;
        }
        __syncwarp();                                           // a key's 8 threads share a warp
#pragma unroll 4
        for (int i = 0; i < BM; ++i) {
            const float p = S.P[gi][key][i], ds = S.S[gi][key][i];
#pragma unroll
            for (int c = 0; c < CV; ++c) {
                const float4 ov = *reinterpret_cast<const float4*>(&S.dO[gi][i][sub * 4 + 32 * c]);
                const float4 qv = *reinterpret_cast<const float4*>(&S.Q[gi][i][sub * 4 + 32 * c]);
                dv[c].x = fmaf(p, ov.x, dv[c].x); dv[c].y = fmaf(p, ov.y, dv[c].y);
                dv[c].z = fmaf(p, ov.z, dv[c].z); dv[c].w = fmaf(p, ov.w, dv[c].w);
                dk[c].x = fmaf(ds, qv.x, dk[c].x); dk[c].y = fmaf(ds, qv.y, dk[c].y);
                dk[c].z = fmaf(ds, qv.z, dk[c].z); dk[c].w = fmaf(ds, qv.w, dk[c].w);
            }
        }
    }
    // The groups' parts meet over their Q and dO tiles.
    __syncthreads();
    float(*pk)[KN][D] = reinterpret_cast<float(*)[KN][D]>(&S.Q[0][0][0]);
    float(*pv)[KN][D] = reinterpret_cast<float(*)[KN][D]>(&S.dO[0][0][0]);
#pragma unroll
    for (int c = 0; c < CV; ++c) {
        *reinterpret_cast<float4*>(&pk[gi][key][sub * 4 + 32 * c]) = dk[c];
        *reinterpret_cast<float4*>(&pv[gi][key][sub * 4 + 32 * c]) = dv[c];
    }
    __syncthreads();
    const int32_t pp = a.bt[lp];
    if (pp < 0 || pp >= a.num_phys) return;                     // recorded by load_key_tile
    const size_t off = (((size_t)pp * a.Hkv + kvh) * a.P + (size_t)(k0 - lp * a.P)) * D;
    for (int i = threadIdx.x; i < n * D; i += GT) {
        const int r = i / D, c = i % D;
        a.dkpool[off + i] = fmaf((pk[0][r][c] + pk[1][r][c]) + (pk[2][r][c] + pk[3][r][c]), scale, a.dkpool[off + i]);
        a.dvpool[off + i] += (pv[0][r][c] + pv[1][r][c]) + (pv[2][r][c] + pv[3][r][c]);
    }
}

template <typename T, int D>
cudaError_t fwd_launch(const AttnArgs& a, cudaStream_t s) {
    static SmemGrant allowed;
    const cudaError_t e = allow_smem(fwd_mod_simt<T, D>, sizeof(FwdSmem<T, D>), allowed);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)row_tiles(a), a.Hkv, a.splits);
    ProfScope ps("fwd_mod_simt", s);
    fwd_mod_simt<T, D><<<grid, NT, sizeof(FwdSmem<T, D>), s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd_launch(const AttnArgs& a, cudaStream_t s) {
    static SmemGrant allowed[2];
    cudaError_t e = allow_smem(bwd_dq_mod_simt<T, D>, sizeof(DqSmem<T, D>), allowed[0]);
    if (e == cudaSuccess) e = allow_smem(bwd_dkdv_mod_simt<T, D>, sizeof(DkvSmem<T, D>), allowed[1]);
    if (e != cudaSuccess) return e;
    {
        ProfScope ps("bwd_dq_mod_simt", s);
        bwd_dq_mod_simt<T, D><<<dim3((unsigned)row_tiles(a), a.Hkv), GT, sizeof(DqSmem<T, D>), s>>>(a);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ProfScope ps("bwd_dkdv_mod_simt", s);
    bwd_dkdv_mod_simt<T, D><<<dim3((unsigned)((a.m.n_keys + KN - 1) / KN), a.Hkv), GT, sizeof(DkvSmem<T, D>), s>>>(
        a, row_tiles(a));
    return cudaGetLastError();
}

}  // namespace

int attn_fwd_mod_simt_splits(const AttnArgs& a) {
    if (a.sel) return 1;
    // Few row tiles leave SMs idle: about two CTAs per SM, each with a key tile at least.
    const int sms = sm_count();
    const int64_t ctas = row_tiles(a) * a.Hkv;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(a.m.n_keys + BN - 1) / BN, 2 * (int64_t)sms / ctas, 128}));
}

cudaError_t launch_attn_fwd_mod_simt(const AttnArgs& a, cudaStream_t s) {
    if (a.dtype == PKV_BF16)
        return a.d == 128 ? fwd_launch<__nv_bfloat16, 128>(a, s) : fwd_launch<__nv_bfloat16, 64>(a, s);
    return a.d == 128 ? fwd_launch<float, 128>(a, s) : fwd_launch<float, 64>(a, s);
}

cudaError_t launch_attn_bwd_mod_simt(const AttnArgs& a, cudaStream_t s) {
    if (a.P % KN) return cudaErrorInvalidValue;
    if (a.dtype == PKV_BF16)
        return a.d == 128 ? bwd_launch<__nv_bfloat16, 128>(a, s) : bwd_launch<__nv_bfloat16, 64>(a, s);
    return a.d == 128 ? bwd_launch<float, 128>(a, s) : bwd_launch<float, 64>(a, s);
}

}  // namespace pkv
