// Linear attention with a decay per head (lin.cuh) on the tensor cores: bf16
// inputs, fp32 accumulators in tensor memory, chunks of 128 rows.
//
// Three launches forward: the chunks' sums of k v^T (lin_part_tc_kernel), the scan
// that turns them into the states before the chunks (lin_scan_bf16_kernel), the
// rows O (lin_rows_tc_kernel). The backward forms both sums and both scans, then
// the rows dQ (the same kernel) and the columns dV and dK (lin_cols_tc_kernel).
//
// Roundings to bf16, beside the outputs': the weighted scores of a chunk and the
// states before (after) a chunk, each once, as operands of products. Sums and
// scans stay in fp32: a weighted operand of the sums is given to the tensor core
// as three bf16 terms that add up to it (24 bits).
#include <cuda_bf16.h>

#include <algorithm>

#include "lin.cuh"
#include "tc.cuh"

namespace pkv {
namespace {

constexpr int kL = kLinTcChunk;
static_assert(kL == 128, "a chunk is the 128 rows of an accumulator");

// 32 bytes to global memory, 32-byte aligned (whole sectors), or as two halves.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// D columns of this thread's accumulator row, times f, to a bf16 row.
template <int D> __device__ __forceinline__ void store_row(uint32_t tmem, float f, __nv_bfloat16* row, bool live, bool wide) {
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + c, r);
        tc::tmem_wait_ld(r);
        if (live)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = pack_bf16x2(__uint_as_float(r[16 * v + 2 * e]) * f, __uint_as_float(r[16 * v + 2 * e + 1]) * f);
                store32(row + c + 16 * v, w, wide);
            }
    }
}

// D columns of this thread's accumulator row, times f, in place.
template <int D> __device__ __forceinline__ void scale_row(uint32_t tmem, float f) {
#pragma unroll
    for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + c, r);
        tc::tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
        tc::tmem_st32(tmem + c, r);
    }
}

// Zeroes rows [m, 128) of a 128-row tile of D / 64 blocks, by `threads` threads:
// what lies behind a sequence may be anything, and 0 * NaN is NaN.
template <int D> __device__ __forceinline__ void zero_tail(uint8_t* tile, int m, int t, int threads) {
    const int n = (kL - m) * 8;
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
        for (int i = t; i < n; i += threads) *reinterpret_cast<uint4*>(tile + b * 16384 + m * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ sums of a chunk

constexpr int kPartStages = 3, kPartRows = 32, kPartWarps = 8;
constexpr int kPartThreads = (kPartWarps + 1) * 32;

template <int D> struct PartLayout {
    static constexpr uint32_t kBlock = kPartRows * 128;              // 64 columns of a stage's rows
    static constexpr uint32_t kOp = D / 64 * kBlock;                 // one operand
    static constexpr uint32_t kStage = 4 * kOp;                      // three terms of A, R
    static constexpr uint32_t kSmem = kPartStages * kStage + 1024;
    static constexpr uint32_t kCols = 128;                           // tensor memory
};

// x's three bf16 terms: hi, what hi leaves, what both leave (packed pairs).
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16x2(x, y);
    x -= bf16lo(hi);
    y -= bf16hi(hi);
    mid = pack_bf16x2(x, y);
    lo = pack_bf16x2(x - bf16lo(mid), y - bf16hi(mid));
}

// part[f][h] = sum_t w_t a_t r_t^T: z 0, k v^T with w = l^(m-1-t); z 1, scale q do^T
// over the group's heads with w = l^(t+1). Eight warps load 32 rows at a time,
// weight and split A and lay both operands out; the ninth issues the products
// (both operands MN-major: the rows are the inner dimension). D = 64 packs two
// terms into the 128 rows of an instruction: accumulator rows 0 .. 63 hold hi's
// sum and, 64 columns on, lo's; rows 64 .. 127 mid's.
template <int D>
__global__ void __launch_bounds__(kPartThreads, 2) lin_part_tc_kernel(const LinArgs a, int z0) {
    using L = PartLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kPartStages], empty[kPartStages], done;
    __shared__ uint32_t tmem_base;
    __shared__ float w[kL];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, h = blockIdx.y;
    const bool grad = blockIdx.z + z0;
    LinChunk c;
    if (!lin_chunk<kL>(a, blockIdx.x, c)) return;
    const int g = grad ? a.Hq / a.Hkv : 1;
    const int per_head = (c.rows + kPartRows - 1) / kPartRows, n_st = per_head * g;
    if (threadIdx.x < kL) {
        const int t = threadIdx.x;
        const float g2 = lin_g2(a, h);
        w[t] = t >= c.rows ? 0.f : grad ? rsqrtf((float)D) * lin_pow(g2, t + 1) : lin_pow(g2, c.rows - 1 - t);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPartStages; ++s) {
            tc::mbar_init(&full[s], kPartWarps * 32);
            tc::mbar_init(&empty[s], 1);
        }
        tc::mbar_init(&done, 1);
        tc::fence_barrier_init();
    }
    if (warp == kPartWarps) {
        tc::tmem_alloc(&tmem_base, L::kCols);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_base;
    if (warp == kPartWarps) {
        const bool leader = tc::elect_one_sync();
        bool ok = true;
        const uint32_t idesc = tc::idesc_bf16(128, D, true, true);
        for (int i = 0; i < n_st; ++i) {
            const int s = i % kPartStages;
            if (!tc::warp_wait(&full[s], (i / kPartStages) & 1, a.wait_err)) { ok = false; break; }
            tc::tc_fence_after();
            const uint32_t base = tc::smem_u32(smem + s * L::kStage);
            const uint64_t r0 = tc::sdesc(base + 3 * L::kOp, L::kBlock, 1024);
            if (leader) {
                if constexpr (D == 128) {
#pragma unroll
                    for (int t = 0; t < 3; ++t)
#pragma unroll
                        for (int k = 0; k < kPartRows / 16; ++k)
                            tc::mma_bf16(tmem, tc::sdesc(base + t * L::kOp + k * 2048, L::kBlock, 1024), tc::sdesc_at(r0, k * 2048),
                                         idesc, (i | t | k) ? 1u : 0u);
                } else {
                    // Blocks hi, mid, then lo and (its sums unused) R.
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < kPartRows / 16; ++k)
                            tc::mma_bf16(tmem + 64 * t, tc::sdesc(base + 2 * t * L::kOp + k * 2048, L::kBlock, 1024),
                                         tc::sdesc_at(r0, k * 2048), idesc, (i | k) ? 1u : 0u);
                }
                tc::mma_commit(&empty[s]);
            }
            __syncwarp();
        }
        if (leader) {
            tc::mma_commit(&done);
            tc::drain_wait(&done, 0);
        }
        __syncwarp();
        (void)ok;
    } else {
        constexpr int VPR = D / 8, NV = kPartRows * VPR / (kPartWarps * 32);      // 16-byte vectors a thread: 2 or 1
        const LinRows &xa = grad ? a.q : a.k, &xr = grad ? a.dout : a.v;
        uint4 ua[2][NV], ur[2][NV];
        auto fetch = [&](int i, uint4 (&da)[NV], uint4 (&dr)[NV]) {
            const int head = grad ? h * g + i / per_head : h, t0 = i % per_head * kPartRows;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int id = threadIdx.x + v * kPartWarps * 32, t = t0 + id / VPR, col = id % VPR * 8;
                da[v] = dr[v] = make_uint4(0, 0, 0, 0);
                if (t < c.rows) {
                    da[v] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(xa.p) + (c.row0 + t) * xa.stride + head * D + col));
                    dr[v] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(xr.p) + (c.row0 + t) * xr.stride + head * D + col));
                }
            }
        };
        bool ok = true;
        auto put = [&](int i, const uint4 (&da)[NV], const uint4 (&dr)[NV]) {
            const int s = i % kPartStages;
            if (i >= kPartStages && ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&empty[s], ((i / kPartStages) - 1) & 1, a.wait_err));
            if (!ok) return;
            uint8_t* st = smem + s * L::kStage;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int id = threadIdx.x + v * kPartWarps * 32, t = id / VPR, col = id % VPR;
                const uint32_t at = col / 8 * L::kBlock + tc::sw128_offset(t, col % 8);
                const float wt = w[i % per_head * kPartRows + t];
                float f[8];
                widen16<__nv_bfloat16>(da[v], f);
                uint4 hi, mid, lo;
                split3(f[0] * wt, f[1] * wt, hi.x, mid.x, lo.x);
                split3(f[2] * wt, f[3] * wt, hi.y, mid.y, lo.y);
                split3(f[4] * wt, f[5] * wt, hi.z, mid.z, lo.z);
                split3(f[6] * wt, f[7] * wt, hi.w, mid.w, lo.w);
                *reinterpret_cast<uint4*>(st + at) = hi;
                *reinterpret_cast<uint4*>(st + L::kOp + at) = mid;
                *reinterpret_cast<uint4*>(st + 2 * L::kOp + at) = lo;
                *reinterpret_cast<uint4*>(st + 3 * L::kOp + at) = dr[v];
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&full[s]);
        };
        fetch(0, ua[0], ur[0]);
        if (n_st > 1) fetch(1, ua[1], ur[1]);
        for (int i = 0; i < n_st; i += 2) {
            put(i, ua[0], ur[0]);
            if (i + 2 < n_st) fetch(i + 2, ua[0], ur[0]);
            if (i + 1 < n_st) put(i + 1, ua[1], ur[1]);
            if (i + 3 < n_st) fetch(i + 3, ua[1], ur[1]);
        }
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&done, 0, a.wait_err));
        tc::tc_fence_after();
        float* out = (grad ? a.gpart : a.part) + ((size_t)blockIdx.x * a.Hkv + h) * D * D;
        const uint32_t base = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        const int row = warp % 4 * 32 + lane;
        if constexpr (D == 128) {
            if (ok)
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    const int col = warp / 4 * 64 + cc * 32;
                    uint32_t r[32];
                    tc::tmem_ld32(base + col, r);
                    tc::tmem_wait_ld(r);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t q[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) q[e] = r[8 * v + e];
                        store32(out + (size_t)row * D + col + 8 * v, q, true);
                    }
                }
        } else {
            // mid's sums cross from rows 64 .. 127 through shared memory (the stages are free by now).
            float* x = reinterpret_cast<float*>(smem);           // [64][65]
            uint32_t r[32], q[32];
            const int col = warp / 4 * 32;
            tc::tmem_ld32(base + col, r);
            tc::tmem_ld32(base + 64 + col, q);
            tc::tmem_wait_ld(r);
            tc::tmem_wait_ld(q);
            if (row >= 64)
#pragma unroll
                for (int e = 0; e < 32; ++e) x[(row - 64) * 65 + col + e] = __uint_as_float(r[e]);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (ok && row < 64)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    uint32_t s[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[e] = __float_as_uint(__uint_as_float(r[8 * v + e]) +
                                               (x[row * 65 + col + 8 * v + e] + __uint_as_float(q[8 * v + e])));
                    store32(out + (size_t)row * D + col + 8 * v, s, true);
                }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kPartWarps) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, L::kCols);
    }
}

// ------------------------------------------------------------------ scan

constexpr int kScanThreads = 128, kScanAhead = 8;

// From a sequence's chunk sums to the states before its chunks (z 0, in order) or
// the gradients of the states after them (z 1, in reverse), in fp32; the kernels
// that multiply by them get them in bf16. A thread owns four elements all along
// (so slot_in may be slot_out) and loads kScanAhead chunks' sums at once.
template <int D>
__global__ void __launch_bounds__(kScanThreads) lin_scan_bf16_kernel(const LinArgs a, int z0, bool keep) {
    constexpr int V = D * D / 4;
    const bool grad = blockIdx.y + z0;
    const int64_t unit = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
    const int e = (int)(unit % V), h = (int)(unit / V % a.Hkv);
    const int64_t b = unit / V / a.Hkv;
    int64_t lo, hi;
    if (!lin_range(a, b, lo, hi)) return;
    const float g2 = lin_g2(a, h), lfull = lin_pow(g2, kL);
    const int64_t first = lin_slot(a, grad ? a.slot_out : a.slot_in, b);
    const int64_t last = lin_slot(a, grad ? a.slot_in : a.slot_out, b);
    float* store = grad ? a.dstate : a.state;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first >= 0) s = reinterpret_cast<const float4*>(store + ((size_t)first * a.Hkv + h) * D * D)[e];
    const int64_t nc = (hi - lo + kL - 1) / kL, f0 = lo / kL + b;
    const float4* part = reinterpret_cast<const float4*>(grad ? a.gpart : a.part);
    uint2* out = reinterpret_cast<uint2*>(grad ? a.gbf : a.sbf);
    const int64_t step = grad ? -1 : 1, at0 = grad ? nc - 1 : 0;
    for (int64_t i = 0; i < nc; i += kScanAhead) {
        const int m = (int)min64(kScanAhead, nc - i);
        float4 x[kScanAhead];
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u)
            if (u < m) x[u] = __ldcs(part + ((size_t)(f0 + at0 + (i + u) * step) * a.Hkv + h) * V + e);
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u)
            if (u < m) {
                const int64_t c = at0 + (i + u) * step;
                out[((size_t)(f0 + c) * a.Hkv + h) * V + e] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
                const int64_t rows = hi - lo - c * kL;
                const float l = rows >= kL ? lfull : lin_pow(g2, (int)rows);
                s.x = fmaf(l, s.x, x[u].x); s.y = fmaf(l, s.y, x[u].y);
                s.z = fmaf(l, s.z, x[u].z); s.w = fmaf(l, s.w, x[u].w);
            }
    }
    if (last >= 0 && (grad || keep)) reinterpret_cast<float4*>(store + ((size_t)last * a.Hkv + h) * D * D)[e] = s;
}

// ------------------------------------------------------------------ rows

// Shared memory of the rows kernel: a ring of (C, S) pairs, R, and a ring of X tiles.
template <int D> struct RowsLayout {
    static constexpr uint32_t kTile = D / 64 * 16384;                // 128 rows
    static constexpr uint32_t kState = D / 64 * D * 128;             // D rows
    static constexpr int kPairs = 2, kX = 2;
    static constexpr uint32_t kOffS = kTile, kPair = kTile + kState;
    static constexpr uint32_t kOffR = kPairs * kPair, kOffX = kOffR + kTile;
    static constexpr uint32_t kSmem = kOffX + kX * kTile + 1024;
};
constexpr int kRowsThreads = 320;

struct RowsBarriers {
    uint64_t pair_full[2], pair_empty[2], r_full, r_empty, x_full[2], x_empty[2];
    uint64_t s_full[2], p_full[2], o_full[2], o_free[2];             // by warpgroup
    uint64_t drain;
    uint32_t tmem_base;
};

// The heads of a CTA: numbers [idx, end) of (chunk, KV head, query head of the
// group), each role of the kernel walking them for itself.
struct HeadWalk {
    const LinArgs& a;
    int64_t idx, end, unit = -1;
    int g, it = -1, pair = -1, f = 0, h = 0, head = 0;
    bool first = false, live = false;
    LinChunk c{};

    __device__ __forceinline__ HeadWalk(const LinArgs& args, int64_t from, int64_t to) : a(args), idx(from - 1), end(to), g(args.Hq / args.Hkv) {}
    // The next head: it counts heads, pair (chunk, KV head)s; first: the first head of its pair here.
    __device__ __forceinline__ bool next() {
        while (++idx < end) {
            const int64_t u = idx / g;
            first = u != unit;
            if (first) {
                unit = u;
                f = (int)(u / a.Hkv);
                h = (int)(u - (int64_t)f * a.Hkv);
                live = lin_chunk<kL>(a, f, c);
                pair += live;
            }
            if (!live) {
                idx = (u + 1) * g - 1;
                continue;
            }
            ++it;
            head = h * g + (int)(idx - u * g);
            return true;
        }
        return false;
    }
};

// out = scale [((X C^T) o M) R + diag(l^(i+1)) X S']. O: X, C, R, S' = Q, K, V, S;
// dQ (GRAD): dO, V, K, S^T. A persistent CTA takes a run of heads. Warp 0 loads
// (TMA), warp 1 issues the products, two warpgroups take the heads in turn, each
// with 256 columns of tensor memory of its own: scores [0, 128), which the
// weighted scores in bf16 overwrite as the A operand of the second product, and
// the output [128, 128 + D), which is X S' first and is scaled by l^(i+1) there
// before the second product adds to it.
// Weights l^(i-j): for 32 x 32 blocks under the diagonal l^(i - 32 b - 31) (one per
// row and block) times l^(31 - (j - 32 b)), both with exponents >= 0; on it from a table.
template <int D, bool GRAD>
__global__ void __launch_bounds__(kRowsThreads, 1)
lin_rows_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_c,
                   const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_s, const LinArgs a,
                   int64_t heads, int wide) {
    using L = RowsLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) RowsBarriers B;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t from = heads * blockIdx.x / gridDim.x, to = heads * (blockIdx.x + 1) / gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&B.pair_full[s], 1);
            tc::mbar_init(&B.pair_empty[s], 1);
            tc::mbar_init(&B.x_full[s], 1);
            tc::mbar_init(&B.x_empty[s], 1);
            tc::mbar_init(&B.s_full[s], 1);
            tc::mbar_init(&B.p_full[s], 128);
            tc::mbar_init(&B.o_full[s], 1);
            tc::mbar_init(&B.o_free[s], 128);
        }
        tc::mbar_init(&B.r_full, 1);
        tc::mbar_init(&B.r_empty, 1);
        tc::mbar_init(&B.drain, 1);
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&B.tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = B.tmem_base;
    HeadWalk w(a, from, to);
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            tc::prefetch_tmap(&map_x);
            tc::prefetch_tmap(&map_c);
            tc::prefetch_tmap(&map_r);
            tc::prefetch_tmap(&map_s);
        }
        bool ok = true;
        int n_x = 0, n_pair = 0, n_r = 0;
        while (w.next()) {
            const int row = (int)w.c.row0;
            if (w.first) {
                const int s = w.pair & 1;
                if (w.pair >= 2 && !tc::warp_wait(&B.pair_empty[s], ((w.pair >> 1) - 1) & 1, a.wait_err)) { ok = false; break; }
                if (lane == 0) {
                    uint8_t* dst = smem + s * L::kPair;
                    tc::mbar_arrive_expect_tx(&B.pair_full[s], L::kPair);
#pragma unroll
                    for (int b = 0; b < D / 64; ++b) {
                        tc::tma_load_3d(dst + b * 16384, &map_c, &B.pair_full[s], 64 * b, w.h, row);
                        tc::tma_load_2d(dst + L::kOffS + b * (D * 128), &map_s, &B.pair_full[s], 64 * b, (w.f * a.Hkv + w.h) * D);
                    }
                }
                n_pair = w.pair + 1;
            }
            {
                const int s = w.it & 1;
                if (w.it >= 2 && !tc::warp_wait(&B.x_empty[s], ((w.it >> 1) - 1) & 1, a.wait_err)) { ok = false; break; }
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&B.x_full[s], L::kTile);
#pragma unroll
                    for (int b = 0; b < D / 64; ++b)
                        tc::tma_load_3d(smem + L::kOffX + s * L::kTile + b * 16384, &map_x, &B.x_full[s], 64 * b, w.head, row);
                }
                n_x = w.it + 1;
            }
            if (w.first) {
                if (w.pair >= 1 && !tc::warp_wait(&B.r_empty, (w.pair - 1) & 1, a.wait_err)) { ok = false; break; }
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&B.r_full, L::kTile);
#pragma unroll
                    for (int b = 0; b < D / 64; ++b)
                        tc::tma_load_3d(smem + L::kOffR + b * 16384, &map_r, &B.r_full, 64 * b, w.h, row);
                }
                n_r = w.pair + 1;
            }
        }
        // None of this CTA's copies may still be landing when it exits.
        if (lane == 0) {
            for (int i = max(0, n_x - 2); i < n_x; ++i) tc::drain_wait(&B.x_full[i & 1], (i >> 1) & 1);
            for (int i = max(0, n_pair - 2); i < n_pair; ++i) tc::drain_wait(&B.pair_full[i & 1], (i >> 1) & 1);
            if (n_r > 0) tc::drain_wait(&B.r_full, (n_r - 1) & 1);
        }
        (void)ok;
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool leader = tc::elect_one_sync();
        const uint32_t idesc_x = tc::idesc_bf16(128, 128, false, false);         // X C^T
        const uint32_t idesc_s = tc::idesc_bf16(128, D, false, !GRAD);           // X S (S [inner][columns]) or X S^T
        const uint32_t idesc_r = tc::idesc_bf16(128, D, false, true);            // P R
        const uint32_t sm = tc::smem_u32(smem);
        const uint64_t dr = tc::sdesc(sm + L::kOffR, 16384, 1024);
        // The second product of head i; `last`: the last one that reads this R.
        auto second = [&](int i, int pair, bool last) -> bool {
            if (!tc::warp_wait(&B.p_full[i & 1], (i >> 1) & 1, a.wait_err)) return false;
            if (!tc::warp_wait(&B.r_full, pair & 1, a.wait_err)) return false;
            tc::tc_fence_after();
            if (leader) {
                const uint32_t t = tmem + (i & 1) * 256;
#pragma unroll
                for (int k = 0; k < 8; ++k) tc::mma_bf16_ts(t + 128, t + k * 8, tc::sdesc_at(dr, k * 2048), idesc_r, 1u);
                tc::mma_commit(&B.o_full[i & 1]);
                if (last) tc::mma_commit(&B.r_empty);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        int prev_pair = -1;
        while (w.next()) {
            const int i = w.it, s = i & 1, ps = w.pair & 1;
            if (w.first && w.pair > 0) {         // the pair before is through with C and S
                if (leader) tc::mma_commit(&B.pair_empty[ps ^ 1]);
                __syncwarp();
            }
            if (w.first && !tc::warp_wait(&B.pair_full[ps], (w.pair >> 1) & 1, a.wait_err)) { ok = false; break; }
            if (!tc::warp_wait(&B.x_full[s], (i >> 1) & 1, a.wait_err)) { ok = false; break; }
            if (i >= 2 && !tc::warp_wait(&B.o_free[s], ((i >> 1) - 1) & 1, a.wait_err)) { ok = false; break; }
            tc::tc_fence_after();
            if (leader) {
                const uint64_t dx = tc::sdesc(sm + L::kOffX + s * L::kTile, 16, 1024);
                const uint64_t dc = tc::sdesc(sm + ps * L::kPair, 16, 1024);
                const uint64_t ds = GRAD ? tc::sdesc(sm + ps * L::kPair + L::kOffS, 16, 1024)
                                         : tc::sdesc(sm + ps * L::kPair + L::kOffS, D * 128, 1024);
                const uint32_t t = tmem + s * 256;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
                    tc::mma_bf16(t, tc::sdesc_at(dx, at), tc::sdesc_at(dc, at), idesc_x, k > 0);
                }
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_bf16(t + 128, tc::sdesc_at(dx, (k >> 2) * 16384 + (k & 3) * 32),
                                 tc::sdesc_at(ds, GRAD ? (k >> 2) * (D * 128) + (k & 3) * 32 : k * 2048), idesc_s, k > 0);
                tc::mma_commit(&B.s_full[s]);
                tc::mma_commit(&B.x_empty[s]);
            }
            __syncwarp();
            if (i > 0 && !second(i - 1, prev_pair, w.first)) { ok = false; break; }
            prev_pair = w.pair;
        }
        if (ok && w.it >= 0) second(w.it, prev_pair, false);
        if (leader) {                            // nothing of ours may still run on the tensor core at exit
            tc::mma_commit(&B.drain);
            tc::drain_wait(&B.drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ weights and outputs
        const int wg = (warp - 2) >> 2, quad = warp & 3, i = quad * 32 + lane;   // row of the chunk
        const int t128 = (threadIdx.x - 64) & 127;
        const uint32_t t = tmem + ((uint32_t)(quad * 32) << 16) + wg * 256;
        const float scale = rsqrtf((float)D);
        const LinRows& out = GRAD ? a.dq : a.o;
        // l's powers, kept while the KV head stays; each warpgroup has tables of its own:
        // l^(x - 31) for x >= 31, else 0, and l^(31 - x).
        __shared__ float diag[2][64], up[2][32];
        int h_of = -1;
        float rb[3], li1 = 0.f;
        bool ok = true;
        while (w.next()) {
            if (w.h != h_of) {
                h_of = w.h;
                const float g2 = lin_g2(a, w.h);
                asm volatile("bar.sync %0, 128;" :: "r"(1 + wg) : "memory");     // nobody reads the old table any more
                if (t128 < 64) diag[wg][t128] = t128 >= 31 ? lin_pow(g2, t128 - 31) : 0.f;
                else if (t128 < 96) up[wg][t128 - 64] = lin_pow(g2, 95 - t128);
#pragma unroll
                for (int b = 0; b < 3; ++b) rb[b] = b < quad ? lin_pow(g2, i - 32 * b - 31) : 0.f;
                li1 = lin_pow(g2, i + 1);
                asm volatile("bar.sync %0, 128;" :: "r"(1 + wg) : "memory");
            }
            // (After a failed wait the walk goes on, only to keep meeting the other warps at the barriers.)
            if ((w.it & 1) != wg || !ok) continue;
            const uint32_t ph = (w.it >> 1) & 1;
            if (w.first && w.c.rows < kL) {      // what lies behind the sequence may be anything
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.r_full, w.pair & 1, a.wait_err));
                if (ok) zero_tail<D>(smem + L::kOffR, w.c.rows, t128, 128);
                tc::fence_proxy_async_smem();
            }
            if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.s_full[wg], ph, a.wait_err));
            if (!ok) continue;
            tc::tc_fence_after();
            uint32_t pk[4][16];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b > quad) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[b][e] = 0u;
                    continue;
                }
                uint32_t r[32];
                tc::tmem_ld32(t + 32 * b, r);
                tc::tmem_wait_ld(r);
                if (b < quad) {
                    const float f = b < 3 ? rb[b < 3 ? b : 0] : 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pk[b][e] = pack_bf16x2(__uint_as_float(r[2 * e]) * (up[wg][2 * e] * f),
                                               __uint_as_float(r[2 * e + 1]) * (up[wg][2 * e + 1] * f));
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float x = 2 * e <= lane ? __uint_as_float(r[2 * e]) * diag[wg][lane - 2 * e + 31] : 0.f;
                        const float y = 2 * e + 1 <= lane ? __uint_as_float(r[2 * e + 1]) * diag[wg][lane - 2 * e + 30] : 0.f;
                        pk[b][e] = pack_bf16x2(x, y);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) tc::tmem_st16(t + 16 * b, pk[b]);
            scale_row<D>(t + 128, li1);
            tc::tmem_wait_st();
            tc::tc_fence_before();
            tc::mbar_arrive(&B.p_full[wg]);
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.o_full[wg], ph, a.wait_err));
            if (!ok) continue;
            tc::tc_fence_after();
            store_row<D>(t + 128, scale, static_cast<__nv_bfloat16*>(out.p) + (w.c.row0 + i) * out.stride + (int64_t)w.head * D,
                         i < w.c.rows, wide);
            tc::tc_fence_before();
            tc::mbar_arrive(&B.o_free[wg]);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ columns

template <int D> struct ColsLayout {
    static constexpr uint32_t kTile = D / 64 * 16384, kState = D / 64 * D * 128;
    static constexpr uint32_t kOffV = kTile, kOffG = 2 * kTile, kOffQ = kOffG + kState, kOffDo = kOffQ + 2 * kTile;
    static constexpr uint32_t kSmem = kOffDo + 2 * kTile + 1024;
    static constexpr uint32_t kColDv = 256, kColDk = 256 + D;
};
constexpr int kColsThreads = 320;

struct ColsBarriers {
    uint64_t kvg_full, q_full[2], do_full[2], q_empty[2], do_empty[2];
    uint64_t q_ready[2], do_ready[2];            // their tails zeroed (a chunk of less than 128 rows)
    uint64_t init_full, init_done, s_full[2], p_full[2], acc_full, drain;
    uint32_t tmem_base;
};

// dV = scale sum_heads ((Q K^T) o M)^T dO + diag(l^(m-1-j)) K G and dK = scale
// sum_heads ((dO V^T) o M)^T Q + diag(l^(m-1-j)) V G^T of one chunk and KV head.
// Scores are formed transposed (keys are the accumulator's rows): K Q^T in
// columns [0, 128) for warpgroup 0 (dV), V dO^T in [128, 256) for warpgroup 1
// (dK); their weighted bf16 values overwrite them as A operands. dV and dK stay
// in tensor memory over all heads; they start as K G and V G^T, scaled there by
// l^(m-1-j) / scale. While one warpgroup weighs its scores the tensor core works
// for the other.
template <int D>
__global__ void __launch_bounds__(kColsThreads, 1)
lin_cols_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                   const __grid_constant__ CUtensorMap map_g, const LinArgs a, int wide) {
    using L = ColsLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) ColsBarriers B;
    __shared__ float diag[64], pw[32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, f = blockIdx.x, h = blockIdx.y;
    LinChunk c;
    if (!lin_chunk<kL>(a, f, c)) return;
    const int g = a.Hq / a.Hkv;
    const bool tail = c.rows < kL;
    const float g2 = lin_g2(a, h);
    if (threadIdx.x < 64) diag[threadIdx.x] = threadIdx.x >= 31 ? lin_pow(g2, threadIdx.x - 31) : 0.f;
    else if (threadIdx.x < 96) pw[threadIdx.x - 64] = lin_pow(g2, threadIdx.x - 64);
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&B.q_full[s], 1);
            tc::mbar_init(&B.do_full[s], 1);
            tc::mbar_init(&B.q_empty[s], 1);
            tc::mbar_init(&B.do_empty[s], 1);
            tc::mbar_init(&B.q_ready[s], 128);
            tc::mbar_init(&B.do_ready[s], 128);
            tc::mbar_init(&B.s_full[s], 1);
            tc::mbar_init(&B.p_full[s], 128);
        }
        tc::mbar_init(&B.kvg_full, 1);
        tc::mbar_init(&B.init_full, 1);
        tc::mbar_init(&B.init_done, 256);
        tc::mbar_init(&B.acc_full, 1);
        tc::mbar_init(&B.drain, 1);
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&B.tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = B.tmem_base;
    if (warp == 0) {
        const int row = (int)c.row0;
        if (lane == 0) {
            tc::mbar_arrive_expect_tx(&B.kvg_full, 2 * L::kTile + L::kState);
#pragma unroll
            for (int b = 0; b < D / 64; ++b) {
                tc::tma_load_3d(smem + b * 16384, &map_k, &B.kvg_full, 64 * b, h, row);
                tc::tma_load_2d(smem + L::kOffG + b * (D * 128), &map_g, &B.kvg_full, 64 * b, (f * a.Hkv + h) * D);
                tc::tma_load_3d(smem + L::kOffV + b * 16384, &map_v, &B.kvg_full, 64 * b, h, row);
            }
        }
        int n = 0;
        for (int i = 0; i < g; ++i) {
            const int s = i & 1;
            if (i >= 2 && !tc::warp_wait(&B.q_empty[s], ((i >> 1) - 1) & 1, a.wait_err)) break;
            if (i >= 2 && !tc::warp_wait(&B.do_empty[s], ((i >> 1) - 1) & 1, a.wait_err)) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&B.q_full[s], L::kTile);
                tc::mbar_arrive_expect_tx(&B.do_full[s], L::kTile);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    tc::tma_load_3d(smem + L::kOffQ + s * L::kTile + b * 16384, &map_q, &B.q_full[s], 64 * b, h * g + i, row);
                    tc::tma_load_3d(smem + L::kOffDo + s * L::kTile + b * 16384, &map_do, &B.do_full[s], 64 * b, h * g + i, row);
                }
            }
            n = i + 1;
        }
        if (lane == 0) {
            tc::drain_wait(&B.kvg_full, 0);
            for (int i = max(0, n - 2); i < n; ++i) {
                tc::drain_wait(&B.q_full[i & 1], (i >> 1) & 1);
                tc::drain_wait(&B.do_full[i & 1], (i >> 1) & 1);
            }
        }
    } else if (warp == 1) {
        const bool leader = tc::elect_one_sync();
        const uint32_t id_s = tc::idesc_bf16(128, 128, false, false), id_acc = tc::idesc_bf16(128, D, false, true);
        const uint32_t id_gt = tc::idesc_bf16(128, D, false, false);
        const uint32_t sm = tc::smem_u32(smem);
        const uint64_t dk = tc::sdesc(sm, 16, 1024), dv = tc::sdesc(sm + L::kOffV, 16, 1024);
        const uint32_t t_dv = tmem + L::kColDv, t_dk = tmem + L::kColDk;
        // Scores K Q^T (x 0) or V dO^T (x 1) of head i.
        auto scores = [&](int i, int x) -> bool {
            const int s = i & 1;
            uint64_t* full = tail ? (x ? B.do_ready : B.q_ready) : (x ? B.do_full : B.q_full);
            if (!tc::warp_wait(&full[s], (i >> 1) & 1, a.wait_err)) return false;
            tc::tc_fence_after();
            if (leader) {
                const uint64_t db = tc::sdesc(sm + (x ? L::kOffDo : L::kOffQ) + s * L::kTile, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
                    tc::mma_bf16(tmem + 128 * x, tc::sdesc_at(x ? dv : dk, at), tc::sdesc_at(db, at), id_s, k > 0);
                }
                tc::mma_commit(&B.s_full[x]);
            }
            __syncwarp();
            return true;
        };
        // dV += P^T dO (x 0) or dK += P'^T Q (x 1) of head i.
        auto add = [&](int i, int x) -> bool {
            const int s = i & 1;
            uint64_t* full = tail ? (x ? B.q_ready : B.do_ready) : (x ? B.q_full : B.do_full);
            if (!tc::warp_wait(&B.p_full[x], i & 1, a.wait_err)) return false;
            if (!tc::warp_wait(&full[s], (i >> 1) & 1, a.wait_err)) return false;
            tc::tc_fence_after();
            if (leader) {
                const uint64_t db = tc::sdesc(sm + (x ? L::kOffQ : L::kOffDo) + s * L::kTile, 16384, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc::mma_bf16_ts(x ? t_dk : t_dv, tmem + 128 * x + k * 8, tc::sdesc_at(db, k * 2048), id_acc, 1u);
                // (the same head's scores of the other kind were issued before: both readers are covered)
                tc::mma_commit(x ? &B.q_empty[s] : &B.do_empty[s]);
            }
            __syncwarp();
            return true;
        };
        bool ok = tc::warp_wait(&B.kvg_full, 0, a.wait_err);
        if (ok) {
            tc::tc_fence_after();
            if (leader) {
                const uint64_t dgn = tc::sdesc(sm + L::kOffG, D * 128, 1024), dgt = tc::sdesc(sm + L::kOffG, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_bf16(t_dv, tc::sdesc_at(dk, (k >> 2) * 16384 + (k & 3) * 32), tc::sdesc_at(dgn, k * 2048), id_acc, k > 0);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_bf16(t_dk, tc::sdesc_at(dv, (k >> 2) * 16384 + (k & 3) * 32),
                                 tc::sdesc_at(dgt, (k >> 2) * (D * 128) + (k & 3) * 32), id_gt, k > 0);
                tc::mma_commit(&B.init_full);
            }
            __syncwarp();
        }
        ok = ok && scores(0, 0) && scores(0, 1);
        ok = ok && tc::warp_wait(&B.init_done, 0, a.wait_err);
        for (int i = 0; ok && i < g; ++i)
            ok = add(i, 0) && (i + 1 >= g || scores(i + 1, 0)) && add(i, 1) && (i + 1 >= g || scores(i + 1, 1));
        if (leader) {
            tc::mma_commit(&B.acc_full);
            tc::drain_wait(&B.acc_full, 0);
        }
        __syncwarp();
    } else {
        const int x = (warp - 2) >> 2, quad = warp & 3, j = quad * 32 + lane;    // key row of the chunk
        const int t128 = (threadIdx.x - 64) & 127;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), acc = lanes + (x ? L::kColDk : L::kColDv), t = lanes + 128 * x;
        const float scale = rsqrtf((float)D);
        // Warpgroup x zeroes the tails of the operand that its own scores do not read as columns alone: Q (0), dO (1).
        auto tails = [&](int i) -> bool {
            const int s = i & 1;
            uint64_t* full = x ? B.do_full : B.q_full;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], (i >> 1) & 1, a.wait_err))) return false;
            zero_tail<D>(smem + (x ? L::kOffDo : L::kOffQ) + s * L::kTile, c.rows, t128, 128);
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(x ? &B.do_ready[s] : &B.q_ready[s]);
            return true;
        };
        float rb[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) rb[b] = b > quad ? lin_pow(g2, 32 * b - j) : 0.f;
        bool ok = !tail || tails(0);
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.init_full, 0, a.wait_err));
        if (ok) {
            tc::tc_fence_after();
            scale_row<D>(acc, j < c.rows ? lin_pow(g2, c.rows - 1 - j) / scale : 0.f);
            tc::tmem_wait_st();
            tc::tc_fence_before();
        }
        tc::mbar_arrive(&B.init_done);
        for (int i = 0; ok && i < g; ++i) {
            if (tail && i + 1 < g && !(ok = tails(i + 1))) break;
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.s_full[x], i & 1, a.wait_err));
            if (!ok) break;
            tc::tc_fence_after();
            uint32_t pk[4][16];
#pragma unroll
            for (int b = 0; b < 4; ++b) {                // queries 32 b ..
                if (b < quad) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[b][e] = 0u;
                    continue;
                }
                uint32_t r[32];
                tc::tmem_ld32(t + 32 * b, r);
                tc::tmem_wait_ld(r);
                const int left = c.rows - 32 * b;
                if (b > quad) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = 2 * e < left ? __uint_as_float(r[2 * e]) * (pw[2 * e] * rb[b]) : 0.f;
                        const float p1 = 2 * e + 1 < left ? __uint_as_float(r[2 * e + 1]) * (pw[2 * e + 1] * rb[b]) : 0.f;
                        pk[b][e] = pack_bf16x2(p0, p1);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = 2 * e >= lane && 2 * e < left ? __uint_as_float(r[2 * e]) * diag[2 * e - lane + 31] : 0.f;
                        const float p1 = 2 * e + 1 >= lane && 2 * e + 1 < left ? __uint_as_float(r[2 * e + 1]) * diag[2 * e + 32 - lane] : 0.f;
                        pk[b][e] = pack_bf16x2(p0, p1);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) tc::tmem_st16(t + 16 * b, pk[b]);
            tc::tmem_wait_st();
            tc::tc_fence_before();
            tc::mbar_arrive(&B.p_full[x]);
        }
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.acc_full, 0, a.wait_err));
        if (ok) {
            tc::tc_fence_after();
            const LinRows& out = x ? a.dk : a.dv;
            store_row<D>(acc, scale, static_cast<__nv_bfloat16*>(out.p) + (c.row0 + j) * out.stride + (int64_t)h * D, j < c.rows, wide >> x & 1);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ launches

bool rows_map(CUtensorMap* m, const LinRows& x, int H, const LinArgs& a, std::string* why) {
    return make_tmap_3d(m, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.d, H, a.n, a.d * 2, x.stride * 2, 64, 1, kL, why);
}
bool states_map(CUtensorMap* m, const void* p, const LinArgs& a, std::string* why) {
    return make_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.d, (uint64_t)a.n_chunks * a.Hkv * a.d, a.d * 2, 64, a.d, why);
}
bool wide_rows(const LinRows& x) { return (reinterpret_cast<uintptr_t>(x.p) & 31) == 0 && x.stride % 16 == 0; }

// Sums z0 .. z0 + nz - 1 (0: k v^T, 1: q do^T) and their scans.
template <int D> cudaError_t states(const LinArgs& a, int z0, int nz, bool keep, cudaStream_t s) {
    static SmemGrant grant;
    cudaError_t e = allow_smem(lin_part_tc_kernel<D>, PartLayout<D>::kSmem, grant);
    if (e != cudaSuccess) return e;
    if (a.n) {
        ProfScope ps("lin_part_tc_kernel", s);
        lin_part_tc_kernel<D><<<dim3(a.n_chunks, a.Hkv, nz), kPartThreads, PartLayout<D>::kSmem, s>>>(a, z0);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    ProfScope ps("lin_scan_bf16_kernel", s);
    lin_scan_bf16_kernel<D><<<dim3((unsigned)(a.n_seq * a.Hkv * (D * D / 4 / kScanThreads)), nz), kScanThreads, 0, s>>>(a, z0, keep);
    return cudaGetLastError();
}

template <int D, bool GRAD> cudaError_t rows(const LinArgs& a, cudaStream_t s, std::string* why) {
    static SmemGrant grant;
    const cudaError_t e = allow_smem(lin_rows_tc_kernel<D, GRAD>, RowsLayout<D>::kSmem, grant);
    if (e != cudaSuccess) return e;
    CUtensorMap x, c, r, st;
    if (!rows_map(&x, GRAD ? a.dout : a.q, a.Hq, a, why) || !rows_map(&c, GRAD ? a.v : a.k, a.Hkv, a, why) ||
        !rows_map(&r, GRAD ? a.k : a.v, a.Hkv, a, why) || !states_map(&st, a.sbf, a, why))
        return cudaErrorInvalidValue;
    const int64_t heads = (int64_t)a.n_chunks * a.Hq;
    const unsigned grid = (unsigned)std::min<int64_t>(heads, sm_count());
    ProfScope ps("lin_rows_tc_kernel", s);
    lin_rows_tc_kernel<D, GRAD><<<grid, kRowsThreads, RowsLayout<D>::kSmem, s>>>(x, c, r, st, a, heads, wide_rows(GRAD ? a.dq : a.o));
    return cudaGetLastError();
}

template <int D> cudaError_t fwd(const LinArgs& a, cudaStream_t s, std::string* why) {
    const cudaError_t e = states<D>(a, 0, 1, true, s);
    return e != cudaSuccess || !a.n ? e : rows<D, false>(a, s, why);
}

template <int D> cudaError_t bwd(const LinArgs& a, cudaStream_t s, std::string* why) {
    cudaError_t e = states<D>(a, 0, 2, false, s);        // the forward's states again, not its result
    if (e == cudaSuccess && a.n) e = rows<D, true>(a, s, why);
    if (e != cudaSuccess || !a.n) return e;
    static SmemGrant grant;
    e = allow_smem(lin_cols_tc_kernel<D>, ColsLayout<D>::kSmem, grant);
    if (e != cudaSuccess) return e;
    CUtensorMap q, k, v, go, gs;
    if (!rows_map(&q, a.q, a.Hq, a, why) || !rows_map(&k, a.k, a.Hkv, a, why) || !rows_map(&v, a.v, a.Hkv, a, why) ||
        !rows_map(&go, a.dout, a.Hq, a, why) || !states_map(&gs, a.gbf, a, why))
        return cudaErrorInvalidValue;
    ProfScope ps("lin_cols_tc_kernel", s);
    lin_cols_tc_kernel<D><<<dim3(a.n_chunks, a.Hkv), kColsThreads, ColsLayout<D>::kSmem, s>>>(
        q, k, v, go, gs, a, (wide_rows(a.dv) ? 1 : 0) | (wide_rows(a.dk) ? 2 : 0));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_fwd_tc(const LinArgs& a, cudaStream_t s, std::string* why) {
    return a.d == 128 ? fwd<128>(a, s, why) : fwd<64>(a, s, why);
}

cudaError_t launch_lin_bwd_tc(const LinArgs& a, cudaStream_t s, std::string* why) {
    return a.d == 128 ? bwd<128>(a, s, why) : bwd<64>(a, s, why);
}

}  // namespace pkv
