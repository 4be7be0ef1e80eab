// Linear attention with a decay per head (lin.cuh) on the tensor cores: bf16
// inputs, fp32 accumulators in tensor memory, chunks of 128 rows.
//
// Three launches forward: the chunks' sums of k v^T (lin_part_tc_kernel), the scan
// that turns them into the states before the chunks (lin_scan_bf16_kernel), the
// rows O (lin_rows_tc_kernel). The backward forms both sums and both scans, then
// the rows dQ (the same kernel) and the columns dV and dK (lin_cols_tc_kernel).
//
// Only the outputs are rounded to bf16. What the tensor core multiplies in bf16 goes there
// as terms that add up: a weighted operand of the sums as three (24 bits, as what they
// add up to stays in fp32 through the scans), the weighted scores of a chunk and the
// states before (after) a chunk as two (16 bits: off by 2^-16 where one term is by 2^-8,
// as much as an output's own rounding). The error of O, dQ, dK and dV against 64 bits is
// that rounding then, 0.0017 relative. TERMS = 1 is the caller's choice
// (PKV_FLAG_LIN_ONE_TERM): 0.0023 to 0.0025, and 10 to 15% less time (4096 rows, 28/4 heads
// of d 128: forward 29.0 us instead of 33.2, both ways 90.2 instead of 105.7).
#include <cuda_bf16.h>

#include <algorithm>

#include "lin.cuh"
#include "mod.cuh"
#include "tc.cuh"

namespace pkv {
namespace {

constexpr int kL = kLinTcChunk;
static_assert(kL == 128, "a chunk is the 128 rows of an accumulator");

// Lets the stream's next kernel start while this one runs, and waits for the ones
// before (their writes are visible then): see launch_after.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Where byte `off` of a box with rows of ROW = 128 (64) bytes and the swizzle of that
// size lies in shared memory (1024-byte aligned base).
template <int ROW> __device__ __forceinline__ uint32_t swizzled(uint32_t off) { return off ^ ((off >> 3) & (ROW == 128 ? 0x70u : 0x30u)); }

// Copies a shared-memory box to global memory (the box unchanged until bulk_wait_read).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(src)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(src)), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// An accumulator's rows lie in the four quadrants of tensor memory, a warp's 32 rows in one.
// In the rows kernel four warps share an accumulator and take half of their rows' columns
// at a time; in the columns kernel eight do, a half of the columns each.

// D / 2 columns of this thread's row, times f, as bf16 pairs.
template <int D> __device__ __forceinline__ void load_half(uint32_t tmem, float f, uint32_t (&o)[D / 4]) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + c, r);
        tc::tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[c / 2 + e] = pack_bf16x2(__uint_as_float(r[2 * e]) * f, __uint_as_float(r[2 * e + 1]) * f);
    }
}

// The warp's 32 rows to global memory: by TMA through `stage` (a thread's own row
// in stores of its own, 32 rows apart from each other, kept the shared-memory
// pipeline from the tensor core: the rows kernel's 24 us became 20), but row by row where the
// sequence ends inside. left: rows of the chunk from this warp's first on. The stage is free.
template <int D>
__device__ __forceinline__ void store_half(const uint32_t (&o)[D / 4], const CUtensorMap* map, uint8_t* stage, int lane, int left,
                                           int column, int head, int64_t row, const LinRows& out) {
    if (left >= 32) {
#pragma unroll
        for (int v = 0; v < D / 16; ++v)
            *reinterpret_cast<uint4*>(stage + swizzled<D>(lane * D + v * 16)) = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, stage, column, head, (int)row);
            tc::bulk_commit();
        }
    } else if (lane < left) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out.p) + (row + lane) * out.stride + (int64_t)head * D + column);
#pragma unroll
        for (int v = 0; v < D / 16; ++v) p[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
    }
}

// D / 2 columns of this thread's row, times f, in place.
template <int D> __device__ __forceinline__ void scale_half(uint32_t tmem, float f) {
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + c, r);
        tc::tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
        tc::tmem_st32(tmem + c, r);
    }
}

// Tensor-memory column, within a tile of scores, of the weighted scores' inner
// indices 16 k .. 16 k + 15, their first (second) terms: each 32 columns are overwritten
// by their own two terms.
__device__ __forceinline__ constexpr uint32_t p_col(int k, int term) { return (k >> 1) * 32 + term * 16 + (k & 1) * 8; }

// Two floats as two bf16 terms each, the nearest and the nearest to what is left, or as the first alone.
template <int TERMS> __device__ __forceinline__ void split(f32x2 p, uint32_t& hi, uint32_t& lo) {
    float x, y;
    unpack2(p, x, y);
    hi = pack_bf16x2(x, y);
    if constexpr (TERMS == 2) {
        unpack2(fma2(pack2(bf16lo(hi), bf16hi(hi)), pack2(-1.f, -1.f), p), x, y);
        lo = pack_bf16x2(x, y);
    }
}

// 32 weighted scores of this thread's row, 16 pairs of first terms and 16 of second ones: pair e
// is put in, all of them stored.
template <int TERMS> __device__ __forceinline__ void put_pair_terms(uint32_t (&pk)[16 * TERMS], int e, f32x2 p) {
    split<TERMS>(p, pk[e], pk[16 * (TERMS - 1) + e]);
}
template <int TERMS> __device__ __forceinline__ void store_block(uint32_t tmem, const uint32_t (&pk)[16 * TERMS]) {
    if constexpr (TERMS == 2) tc::tmem_st32(tmem, pk);
    else tc::tmem_st16(tmem, pk);
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

constexpr int kPartRows = 64, kPartRaw = 5, kPartSplit = 2, kPartWarps = 8;
constexpr int kPartThreads = (2 + kPartWarps + 4) * 32;

template <int D> struct PartLayout {
    static constexpr uint32_t kBlock = kPartRows * 128;              // 64 columns of a stage's rows
    static constexpr uint32_t kOp = D / 64 * kBlock;                 // one operand
    static constexpr uint32_t kRaw = 2 * kOp;                        // A as loaded, R
    static constexpr uint32_t kOffStage = kPartRaw * kRaw;           // a unit's sums, in boxes of 32 x 32
    static constexpr uint32_t kSmem = kOffStage + D * D * 4 + 1024;
    static constexpr uint32_t kColA = 256;                           // tensor memory: A's terms, 128 columns a stage
};

struct PartBarriers {
    uint64_t raw_full[kPartRaw], raw_empty[kPartRaw], split_full[kPartSplit], split_empty[kPartSplit];
    uint64_t acc_full[2], acc_empty[2], drain;
    uint32_t tmem_base;
};

// Three bf16 terms of each of two floats, by truncation: their leading 8 bits, the
// next 8 and the last 8. The differences are exact, so the terms add up to the
// floats (cutting takes fewer instructions than rounding, and the sum is what counts).
__device__ __forceinline__ void split3(f32x2 p, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const f32x2 minus = pack2(-1.f, -1.f);
    auto cut = [&]() -> uint32_t {               // p's leading terms, which leave p
        float x, y;
        unpack2(p, x, y);
        const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
        p = fma2(pack2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u)), minus, p);
        return __byte_perm(u, v, 0x7632);
    };
    hi = cut();
    mid = cut();
    lo = cut();
}

// Heads of the rows kernel for each CTA: laid end to end and cut into one length a CTA,
// `per` each, one more for the first `more`; or (units > 0) whole units of g heads, every
// grid-th from the last one down: all CTAs are at neighbouring chunks then, those first
// whose states the scan wrote last. The former where a unit more or less would show; the
// latter from 8 units a CTA on (16 heads of 32768 rows: 284.6 us instead of 289.0).
struct Cut {
    int per, more, units;
    __device__ __forceinline__ int begin(int g) const {
        return units ? 0 : per * (int)blockIdx.x + min((int)blockIdx.x, more);
    }
    __device__ __forceinline__ int end(int g) const {
        return units ? (units - 1 - (int)blockIdx.x) / (int)gridDim.x * g + g : begin(g) + per + ((int)blockIdx.x < more);
    }
    __device__ __forceinline__ int unit(int q) const { return units ? units - 1 - (int)(blockIdx.x + q * gridDim.x) : q; }
};

// The units of a CTA, chunks of a KV head: numbers blockIdx.x, + gridDim.x, ...; a
// backward's q do^T (g heads of work each) come first, then the k v^T (one each).
// (Units cut by work instead, the short ones on the CTAs that the long ones leave:
// 24 us instead of 20 for a training chunk, as a short unit is mostly latency.)
struct PartWalk {
    const LinArgs& a;
    int per_kind, n, i, it = -1;
    bool both, grad = false;
    int f = 0, h = 0;
    LinChunk c{};
    const LinCuts* cuts;
    __device__ __forceinline__ PartWalk(const LinArgs& args, bool both_, const LinCuts* first)
        : a(args), per_kind(args.n_chunks * args.Hkv), n(both_ ? 2 * per_kind : per_kind), i((int)blockIdx.x - (int)gridDim.x), both(both_),
          cuts(first) {}
    __device__ __forceinline__ bool next() {
        while ((i += gridDim.x) < n) {
            grad = both && i < per_kind;
            const int u = both && !grad ? i - per_kind : i;
            f = u / a.Hkv;
            h = u - f * a.Hkv;
            if (!both) f = a.n_chunks - 1 - f;   // the scan begins with the sums that were written last
            if (!lin_chunk<kL>(a, cuts, f, c)) continue;
            ++it;
            return true;
        }
        return false;
    }
    __device__ __forceinline__ int heads() const { return grad ? a.Hq / a.Hkv : 1; }
    __device__ __forceinline__ int stages() const { return (c.rows + kPartRows - 1) / kPartRows; }
};

// part[f][h] = sum_t w_t a_t r_t^T: k v^T with w = l^(m-1-t), and for a backward
// (both) also scale q do^T over the group's heads with w = l^(t+1). Warp 0 loads
// 64 rows of both operands at a time (TMA). Eight warps weight A, split it into three
// terms and put them into tensor memory, transposed: a thread has one column of A
// (a lane) and 32 rows. Warp 1 issues the products, R (MN-major) from shared memory;
// four warps write sums out. With A's terms in shared memory too, the products' and the
// weighting's traffic there was the bound. Now the weighting is, by its arithmetic: it is
// four fifths of a stage's time, and 16 warps at it were no faster than eight (mean of a
// training chunk's two launches 19.5 us, 18.6 with eight). 4096 rows, 28/4 heads of d 128:
// 10 us, with q do^T 23; 32768 rows of 16 heads: 84 us for 537 MB (6.4 TB/s, HBM's bound).
// The sums of q do^T have an accumulator for the large term and one for the small
// ones: each addition rounds in fp32, and the small terms' would triple their number;
// those of k v^T, of 128 rows alone, have one, and two units alternate between both.
// D = 64 packs two terms into the 128 lanes of an instruction: lanes 0 .. 63 hold hi's
// sum and, 64 columns on, lo's; lanes 64 .. 127 mid's.
template <int D, bool BOTH>
__global__ void __maxnreg__(BOTH ? 128 : 88)
lin_part_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                   const __grid_constant__ CUtensorMap map_kv_out, const __grid_constant__ CUtensorMap map_qdo_out, const LinArgs a) {
    using L = PartLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) PartBarriers B;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPartRaw; ++s) {
            tc::mbar_init(&B.raw_full[s], 1);
            tc::mbar_init(&B.raw_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&B.split_full[s], kPartWarps * 32);
            tc::mbar_init(&B.split_empty[s], 1);
            tc::mbar_init(&B.acc_full[s], 1);
            tc::mbar_init(&B.acc_empty[s], 128);
        }
        tc::mbar_init(&B.drain, 1);
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&B.tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_k);
        tc::prefetch_tmap(&map_v);
        if (BOTH) {
            tc::prefetch_tmap(&map_q);
            tc::prefetch_tmap(&map_do);
        }
    }
    __shared__ LinCuts cuts;
    constexpr int kDecays = 64;
    __shared__ float decays[kDecays];            // log2 of the first KV heads' decays
    if (warp == 2) cuts.load(a);
    for (int h = threadIdx.x - 96; h >= 0 && h < min(a.Hkv, kDecays); h += kPartThreads - 96) decays[h] = lin_g2(a, h);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    PartWalk w(a, BOTH, &cuts);
    bool more = w.next();
    launch_dependents();
    const uint32_t tmem = B.tmem_base;
    int st = 0;                                  // stages so far
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        bool ok = true;
        for (; ok && more; more = w.next()) {
            const int ns = w.stages(), total = w.heads() * ns;
            const CUtensorMap *ma = w.grad ? &map_q : &map_k, *mr = w.grad ? &map_do : &map_v;
            int head = w.grad ? w.h * w.heads() : w.h, row = (int)w.c.row0, left = ns;
            for (int i = 0; i < total; ++i, ++st) {
                const int s = st % kPartRaw;
                if (st >= kPartRaw && !tc::warp_wait(&B.raw_empty[s], (st / kPartRaw - 1) & 1, a.wait_err)) { ok = false; break; }
                if (lane == 0) {
                    uint8_t* dst = smem + s * L::kRaw;
                    tc::mbar_arrive_expect_tx(&B.raw_full[s], L::kRaw);
#pragma unroll
                    for (int b = 0; b < D / 64; ++b) {
                        tc::tma_load_3d(dst + b * L::kBlock, ma, &B.raw_full[s], 64 * b, head, row);
                        tc::tma_load_3d(dst + L::kOp + b * L::kBlock, mr, &B.raw_full[s], 64 * b, head, row);
                    }
                }
                row += kPartRows;
                if (--left == 0) {
                    left = ns;
                    ++head;
                    row = (int)w.c.row0;
                }
            }
        }
        // None of this CTA's copies may still be landing when it exits.
        if (lane == 0)
            for (int i = max(0, st - kPartRaw); i < st; ++i) tc::drain_wait(&B.raw_full[i % kPartRaw], (i / kPartRaw) & 1);
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const bool leader = tc::elect_one_sync();
        const uint32_t idesc = tc::idesc_bf16(128, D, false, true);
        const uint32_t sm = tc::smem_u32(smem);
        bool ok = true;
        int acc = 0;                             // accumulators used so far: number n is columns 128 (n & 1) ..
        for (; ok && more; more = w.next()) {
            const int total = w.heads() * w.stages(), na = D == 128 && w.grad ? 2 : 1;
            for (int n = acc; ok && n < acc + na; ++n)
                ok = n < 2 || tc::warp_wait(&B.acc_empty[n & 1], ((n >> 1) - 1) & 1, a.wait_err);
            if (!ok) break;
            const uint32_t t = tmem + (acc & 1) * 128, t_small = tmem + ((acc + na - 1) & 1) * 128;
            for (int i = 0; i < total; ++i, ++st) {
                const int s = st % kPartRaw, p = st % kPartSplit;
                if (!tc::warp_wait(&B.split_full[p], (st / kPartSplit) & 1, a.wait_err)) { ok = false; break; }
                tc::tc_fence_after();
                if (leader) {
                    const uint64_t r0 = tc::sdesc(sm + s * L::kRaw + L::kOp, L::kBlock, 1024);
                    const uint32_t ta = tmem + L::kColA + p * 128;
                    if constexpr (D == 128) {
#pragma unroll
                        for (int x = 0; x < 3; ++x)
#pragma unroll
                            for (int k = 0; k < kPartRows / 16; ++k)
                                tc::mma_bf16_ts(x ? t_small : t, ta + 32 * x + 8 * k, tc::sdesc_at(r0, k * 2048), idesc,
                                                (i | k | (x == 1 ? na == 1 : x)) ? 1u : 0u);
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x)              // hi and mid, then lo
#pragma unroll
                            for (int k = 0; k < kPartRows / 16; ++k)
                                tc::mma_bf16_ts(t + 64 * x, ta + 32 * x + 8 * k, tc::sdesc_at(r0, k * 2048), idesc, (i | k) ? 1u : 0u);
                    }
                    tc::mma_commit(&B.raw_empty[s]);
                    tc::mma_commit(&B.split_empty[p]);
                    if (i + 1 == total)
                        for (int n = acc; n < acc + na; ++n) tc::mma_commit(&B.acc_full[n & 1]);
                }
                __syncwarp();
            }
            acc += na;
        }
        if (leader) {                            // nothing of ours may still run on the tensor core at exit
            tc::mma_commit(&B.drain);
            tc::drain_wait(&B.drain, 0);
        }
        __syncwarp();
    } else if (warp < 2 + kPartWarps) {
        // ------------------------------------------------------------ weights and terms
        const int tid = threadIdx.x - 64, quad = warp & 3, half = (warp - 2) >> 2;       // rows 32 half .. of a stage
        const int col = (quad * 32 + lane) % D;                                          // A's column; D 64: twice
        const uint32_t base = col / 64 * L::kBlock + half * 4096 + col % 8 * 2;
        const uint32_t chunk = col % 64 / 8;
        const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16) + L::kColA + 16 * half;
        __shared__ __align__(16) float weights[2][kL];
        bool ok = true;
        int unit = 0;
        for (; more; more = w.next(), ++unit) {
            // Weights of units in turn: who is at the second of two barriers has left the first unit's.
            // (After a failed wait the walk goes on, only to keep meeting the other warps here.)
            float* wt = weights[unit & 1];
            const int ns = w.stages(), total = w.heads() * ns, m = w.c.rows;
            if (tid < kL) {
                const float g2 = w.h < kDecays ? decays[w.h] : lin_g2(a, w.h);
                wt[tid] = tid >= m ? 0.f : w.grad ? rsqrtf((float)D) * lin_pow(g2, tid + 1) : lin_pow(g2, m - 1 - tid);
            }
            asm volatile("bar.sync 2, 256;" ::: "memory");
            int q = 0;                           // stage of the chunk
            for (int i = 0; ok && i < total; ++i, ++st, q = q + 1 == ns ? 0 : q + 1) {
                const int s = st % kPartRaw, p = st % kPartSplit;
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.raw_full[s], (st / kPartRaw) & 1, a.wait_err));
                if (!ok) break;
                const uint8_t* raw = smem + s * L::kRaw + base;
                const int left = m - q * kPartRows;
                if (left < kPartRows) {          // behind the sequence: anything, and 0 * NaN is NaN
                    uint8_t* r = smem + s * L::kRaw + L::kOp + left * 128;
                    for (int y = tid; y < (kPartRows - left) * 8 * (D / 64); y += kPartWarps * 32) {
                        const int bl = y / ((kPartRows - left) * 8), at = y % ((kPartRows - left) * 8);
                        *reinterpret_cast<uint4*>(r + bl * L::kBlock + at * 16) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_proxy_async_smem();
                }
                const ulonglong2* wq = reinterpret_cast<const ulonglong2*>(wt + q * kPartRows + 32 * half);
#pragma unroll
                for (int z = 0; z < 2; ++z) {    // 16 rows at a time: few registers leave room for CTAs of the scan, see below
                    uint32_t x[16], hi[8], mid[8], lo[8];
#pragma unroll
                    for (int t = 0; t < 16; ++t) {
                        x[t] = (uint32_t)*reinterpret_cast<const uint16_t*>(raw + (16 * z + t) * 128 + ((chunk ^ (t & 7)) << 4)) << 16;
                        if (left < kPartRows && 32 * half + 16 * z + t >= left) x[t] = 0u;
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const ulonglong2 k = wq[4 * z + t];
                        split3(mul2(pack2(__uint_as_float(x[4 * t]), __uint_as_float(x[4 * t + 1])), k.x), hi[2 * t], mid[2 * t], lo[2 * t]);
                        split3(mul2(pack2(__uint_as_float(x[4 * t + 2]), __uint_as_float(x[4 * t + 3])), k.y), hi[2 * t + 1], mid[2 * t + 1],
                               lo[2 * t + 1]);
                    }
                    // (only now does the place have to be free: products ran meanwhile)
                    if (z == 0 && st >= kPartSplit) {
                        ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.split_empty[p], (st / kPartSplit - 1) & 1, a.wait_err));
                        if (!ok) break;
                        tc::tc_fence_after();
                    }
                    const uint32_t at = ta + p * 128 + 8 * z;
                    if constexpr (D == 128) {
                        tc::tmem_st8(at, hi);
                        tc::tmem_st8(at + 32, mid);
                        tc::tmem_st8(at + 64, lo);
                    } else if (quad < 2) {
                        tc::tmem_st8(at, hi);
                        tc::tmem_st8(at + 32, lo);
                    } else {
                        tc::tmem_st8(at, mid);
                    }
                }
                if (!ok) break;
                tc::tmem_wait_st();
                tc::tc_fence_before();
                tc::mbar_arrive(&B.split_full[p]);
            }
        }
    } else {
        // ------------------------------------------------------------ sums out
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        __shared__ float cross[64][33];          // D 64: mid's sums, 32 columns at a time
        uint8_t* stage = smem + L::kOffStage + quad * (D / 32 * 4096);
        bool ok = true;
        int acc = 0;
        for (; more; more = w.next()) {
            const int na = D == 128 && w.grad ? 2 : 1;
            for (int n = acc; n < acc + na; ++n)
                if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.acc_full[n & 1], (n >> 1) & 1, a.wait_err));
            if (!ok && D == 128) break;
            tc::tc_fence_after();
            const uint32_t t = lanes + (acc & 1) * 128, t_small = lanes + ((acc + 1) & 1) * 128;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t r[32], q[32];
                tc::tmem_ld32(t + c, r);
                if (D == 64) tc::tmem_ld32(t + D + c, q);
                else if (na == 2) tc::tmem_ld32(t_small + c, q);
                else
#pragma unroll
                    for (int e = 0; e < 32; ++e) q[e] = 0u;
                tc::tmem_wait_ld(r);
                tc::tmem_wait_ld(q);
                if (c + 32 == D) {               // all of it is in registers
                    tc::tc_fence_before();
                    for (int n = acc; n < acc + na; ++n) tc::mbar_arrive(&B.acc_empty[n & 1]);
                }
                if constexpr (D == 64) {
                    // (after a failed wait this goes on, only to keep meeting the other warps)
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (row >= 64)
#pragma unroll
                        for (int e = 0; e < 32; ++e) cross[row - 64][e] = __uint_as_float(r[e]);
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (row < 64)
#pragma unroll
                        for (int e = 0; e < 32; ++e) q[e] = __float_as_uint(__uint_as_float(q[e]) + cross[row][e]);
                }
                if (ok && quad * 32 < D) {
                    uint8_t* at = stage + c / 32 * 4096;
                    if (c == 0) {
                        if (lane == 0) tc::bulk_wait_read();                     // the last unit's boxes have left
                        __syncwarp();
                    }
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        float4 x;
                        x.x = __uint_as_float(r[4 * v]) + __uint_as_float(q[4 * v]);
                        x.y = __uint_as_float(r[4 * v + 1]) + __uint_as_float(q[4 * v + 1]);
                        x.z = __uint_as_float(r[4 * v + 2]) + __uint_as_float(q[4 * v + 2]);
                        x.w = __uint_as_float(r[4 * v + 3]) + __uint_as_float(q[4 * v + 3]);
                        *reinterpret_cast<float4*>(at + swizzled<128>(lane * 128 + v * 16)) = x;
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(w.grad ? &map_qdo_out : &map_kv_out, at, c, (w.f * a.Hkv + w.h) * D + quad * 32);
                        tc::bulk_commit();
                    }
                }
            }
            acc += na;
        }
        if (lane == 0) bulk_wait();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ scan

constexpr int kScanThreads = 128, kScanAhead = 16;

// From a sequence's chunk sums to the states before its chunks (y 0, in order) or
// the gradients of the states after them (y 1, in reverse), in fp32. The kernels
// that multiply by them get them as bf16 terms, which take the place of the sums: a row
// of D sums becomes D first terms and D second ones. A row is a warp's (D 64: two are), which
// has read it when it writes. (In memory of their own: 314.6 us instead of 312.0 for a
// forward of 16 heads of 32768 rows, and twice the scratch.) A thread owns four elements all
// along (so slot_in may be slot_out) and has kScanAhead chunks' sums on their way at once:
// what bounds the scan is the latency of these rounds and of what comes before them,
// which overlaps the kernel before where an SM has room beside it. Past L2's size HBM bounds
// it (16 heads of 32768 rows of d 128: 100 us for 537 MB; with one term 76 for 402). More
// chunks at once, or each next one asked for as one is used up, were slower, up to twice
// the time; so were stores marked as streaming (forward of 4096 rows, 28/4 heads: 33.3 us
// instead of 33.0), as the rows kernel reads them next.
template <int D, int TERMS>
__global__ void __launch_bounds__(kScanThreads, 5) lin_scan_bf16_kernel(const LinArgs a) {
    constexpr int V = D * D / 4;
    const bool grad = blockIdx.y;
    const int64_t unit = (int64_t)blockIdx.x * kScanThreads + threadIdx.x;
    const int e = (int)(unit % V);
    const int64_t bh = unit / V, b = bh / a.Hkv;
    const int h = (int)(bh - b * a.Hkv);
    launch_dependents();
    // (a backward scans k v^T for the states alone: the forward has stored the last one)
    const int32_t *from = grad ? a.slot_out : a.slot_in, *to = grad ? a.slot_in : gridDim.y > 1 ? nullptr : a.slot_out;
    const int64_t lo = a.cu ? a.cu[b] : 0, hi = a.cu ? a.cu[b + 1] : a.n;        // all loads before the first check
    const int32_t first_ = from ? from[b] : -1, last_ = to ? to[b] : -1;
    const float g2 = lin_g2(a, h);
    const bool good = lin_good(a, lo, hi);
    const int64_t first = lin_good_slot(a, first_), last = lin_good_slot(a, last_);
    float4* store = reinterpret_cast<float4*>(grad ? a.dstate : a.state);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (good && first >= 0) s = store[((size_t)first * a.Hkv + h) * V + e];      // (older than the kernel before)
    if (blockIdx.x % (V / kScanThreads * a.Hkv) == 0) lin_check_alone(a, to, from, b, last, a.n_seq);
    wait_for_kernels();
    if (!good) return;
    const int nc = (int)((hi - lo + kL - 1) / kL);
    const float lfull = lin_pow(g2, kL), ltail = lin_pow(g2, (int)(hi - lo - (int64_t)(nc - 1) * kL));     // the last chunk's rows
    const int64_t at = ((lo / kL + b + (grad ? nc - 1 : 0)) * a.Hkv + h) * V, step = (int64_t)a.Hkv * V * (grad ? -1 : 1);
    const float4* in = reinterpret_cast<const float4*>(grad ? a.gpart : a.part) + at + e;
    uint2* out = reinterpret_cast<uint2*>((grad ? a.gpart : a.part) + 4 * at) + e / (D / 4) * (D / 2) + e % (D / 4);
    float4* end = last >= 0 ? store + ((size_t)last * a.Hkv + h) * V + e : nullptr;
    for (int i = 0; i < nc; i += kScanAhead) {
        const int m = min(kScanAhead, nc - i);
        float4 x[kScanAhead];
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u) {
            if (u < m) x[u] = __ldcg(in);
            in += step;
        }
        __syncwarp();                            // the warp has read what it overwrites
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u)
            if (u < m) {
                uint2 hi, lo;
                split<TERMS>(pack2(s.x, s.y), hi.x, lo.x);
                split<TERMS>(pack2(s.z, s.w), hi.y, lo.y);
                *out = hi;
                if (TERMS == 2) out[D / 4] = lo;
                out += 2 * step;
                const float l = i + u == (grad ? 0 : nc - 1) ? ltail : lfull;
                s.x = fmaf(l, s.x, x[u].x);
                s.y = fmaf(l, s.y, x[u].y);
                s.z = fmaf(l, s.z, x[u].z);
                s.w = fmaf(l, s.w, x[u].w);
            }
    }
    if (end) *end = s;
}

// ------------------------------------------------------------------ rows

// Shared memory of the rows kernel: C, S (two terms) and R of a (chunk, KV head) pair, an X
// tile for each group of warps, a box of outputs for each warp.
template <int D, int TERMS> struct RowsLayout {
    static constexpr uint32_t kTile = D / 64 * 16384;                // 128 rows
    static constexpr uint32_t kState = D / 64 * D * 128;             // D rows
    static constexpr uint32_t kOffS = kTile, kOffR = kOffS + TERMS * kState, kOffX = kOffR + kTile, kOffStage = kOffX + 2 * kTile;
    static constexpr uint32_t kStage = 32 * D;
    static constexpr uint32_t kSmem = kOffStage + 8 * kStage + 1024;
};
constexpr int kRowsThreads = 3 * 32 + 2 * 128;

struct RowsBarriers {
    uint64_t c_full, st_full, pair_empty, r_full, r_empty;
    // R's tail zeroed, or none (by the group of the pair's first head). Two, in turn: an issuing warp
    // may still have to see a pair's when the other group is at the next pair's; the one after that
    // needs C's place, which both warps give up only after they have seen this one.
    uint64_t r_ready[2];
    uint64_t x_full[2], x_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], o_free[2], drain[2];     // by group
    uint32_t tmem_base;
};

// The heads of a CTA: numbers [idx, end) of (chunk, KV head, query head of the
// group), each role of the kernel walking them for itself.
struct HeadWalk {
    const LinArgs& a;
    Cut cut;
    int g, idx, end, run = -1;                   // run: of g numbers
    int it = -1, pair = -1, f = 0, h = 0, head = 0;
    bool first = false, live = false;
    LinChunk c{};
    const LinCuts* cuts;

    __device__ __forceinline__ HeadWalk(const LinArgs& args, Cut c, const LinCuts* first)
        : a(args), cut(c), g(args.Hq / args.Hkv), idx(c.begin(g) - 1), end(c.end(g)), cuts(first) {}
    // The next head: it counts heads, pair (chunk, KV head)s; first: the first head of its pair here.
    __device__ __forceinline__ bool next() {
        while (++idx < end) {
            if (run < 0 || idx >= (run + 1) * g) {
                run = idx / g;
                const int unit = cut.unit(run);
                f = unit / a.Hkv;
                h = unit - f * a.Hkv;
                live = lin_chunk<kL>(a, cuts, f, c);
                pair += live;
                first = true;
            } else {
                first = false;
            }
            if (!live) {
                idx = (run + 1) * g - 1;
                continue;
            }
            ++it;
            head = h * g + (idx - run * g);
            return true;
        }
        return false;
    }
};

// out = scale [((X C^T) o M) R + diag(l^(i+1)) X S']. O: X, C, R, S' = Q, K, V, S;
// dQ (GRAD): dO, V, K, S^T. A persistent CTA takes a run of heads. Warp 0 loads
// (TMA); two groups of four warps take the heads in turn, each with a warp (1, 2)
// that issues its products and 256 columns of tensor memory of its own: scores
// [0, 128), which the weighted scores' bf16 terms overwrite as the A operand of the
// second product, and the output [128, 128 + D), which is X S' first and is scaled
// by l^(i+1) there before the second product adds to it, in two halves: that of keys
// 0 .. 63 runs while the weights of the others are formed (ragged prompts, 64/8 heads of
// d 64: 39.6 -> 38.4 us). (One issuing warp for both
// made each second product wait for the other group's output to be read: 2.1 us a head.)
// Weights l^(i-j): for 32 x 32 blocks under the diagonal l^(i - 32 b - 31) (one per
// row and block) times l^(31 - (j - 32 b)), both with exponents >= 0; on it from a table.
// What bounds it is a group's chain from a head to its next: X's load, two products and
// their reading and writing in tensor memory, and the store; the tensor pipe is busy for a third
// of the time. 4096 rows, 28/4 heads of d 128: 23 us (six heads a CTA; 71 MB), of which the
// last 14 follow the states; with one term 20. 32768 rows of 16 heads, a state for each:
// 137 us for 805 MB (5.9 TB/s). X asked for further ahead, to L2 or to a second tile a group,
// was slower (one term, both ways of the 4096 rows 95 us instead of 91), as those loads come
// before the kernels that the states still wait for.
template <int D, bool GRAD, int TERMS>
__global__ void __launch_bounds__(kRowsThreads, 1)
lin_rows_tc_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_c,
                   const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_s,
                   const __grid_constant__ CUtensorMap map_out, const LinArgs a, Cut cut) {
    using L = RowsLayout<D, TERMS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) RowsBarriers B;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&B.r_ready[s], 128);
            tc::mbar_init(&B.x_full[s], 1);
            tc::mbar_init(&B.x_empty[s], 1);
            tc::mbar_init(&B.s_full[s], 1);
            tc::mbar_init(&B.p_half[s], 128);
            tc::mbar_init(&B.p_full[s], 128);
            tc::mbar_init(&B.o_full[s], 1);
            tc::mbar_init(&B.o_free[s], 128);
            tc::mbar_init(&B.drain[s], 1);
        }
        tc::mbar_init(&B.c_full, 1);
        tc::mbar_init(&B.st_full, 1);
        tc::mbar_init(&B.pair_empty, 2);
        tc::mbar_init(&B.r_full, 1);
        tc::mbar_init(&B.r_empty, 2);
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&B.tmem_base, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        tc::prefetch_tmap(&map_x);
        tc::prefetch_tmap(&map_c);
        tc::prefetch_tmap(&map_r);
        tc::prefetch_tmap(&map_s);
    }
    __shared__ LinCuts cuts;
    if (warp == 2) cuts.load(a);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    HeadWalk w(a, cut, &cuts);
    bool more = w.next();
    launch_dependents();
    const uint32_t tmem = B.tmem_base;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        bool waited = false;
        int n_x = 0, n_c = 0, n_s = 0, n_r = 0;
        auto tiles = [&](uint32_t at, const CUtensorMap* map, uint64_t* full, int head) {
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) tc::tma_load_3d(smem + at + b * 16384, map, full, 64 * b, head, (int)w.c.row0);
            }
        };
        auto load_x = [&]() {
            tiles(L::kOffX + (w.it & 1) * L::kTile, &map_x, &B.x_full[w.it & 1], w.head);
            n_x = w.it + 1;
        };
        auto load_s = [&](int state) {
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&B.st_full, TERMS * L::kState);
#pragma unroll
                for (int b = 0; b < TERMS * D / 64; ++b) tc::tma_load_2d(smem + L::kOffS + b * (D * 128), &map_s, &B.st_full, 64 * b, state * D);
            }
            ++n_s;
        };
        auto load_c = [&]() {
            tiles(0, &map_c, &B.c_full, w.h);
            ++n_c;
        };
        auto load_r = [&]() {
            tiles(L::kOffR, &map_r, &B.r_full, w.h);
            ++n_r;
        };
        // Until the states are there (the operands are older than the kernels before): the first
        // pair's C and R and the first two heads' X, if both are that pair's.
        if (more) {
            const int state = w.f * a.Hkv + w.h;
            load_c();
            load_x();
            load_r();
            if ((more = w.next()) && !w.first) {
                load_x();
                more = w.next();
            }
            wait_for_kernels();
            waited = true;
            load_s(state);
        }
        for (; more; more = w.next()) {
            if (w.first) {
                if (!tc::warp_wait(&B.pair_empty, (w.pair - 1) & 1, a.wait_err)) break;
                load_c();
            }
            if (w.it >= 2 && !tc::warp_wait(&B.x_empty[w.it & 1], ((w.it >> 1) - 1) & 1, a.wait_err)) break;
            load_x();
            if (w.first) {
                load_s(w.f * a.Hkv + w.h);
                if (!tc::warp_wait(&B.r_empty, (w.pair - 1) & 1, a.wait_err)) break;
                load_r();
            }
        }
        if (!waited) wait_for_kernels();         // a kernel never ends before the one it may overlap
        // None of this CTA's copies may still be landing when it exits.
        if (lane == 0) {
            for (int i = max(0, n_x - 2); i < n_x; ++i) tc::drain_wait(&B.x_full[i & 1], (i >> 1) & 1);
            if (n_c > 0) tc::drain_wait(&B.c_full, (n_c - 1) & 1);
            if (n_s > 0) tc::drain_wait(&B.st_full, (n_s - 1) & 1);
            if (n_r > 0) tc::drain_wait(&B.r_full, (n_r - 1) & 1);
        }
    } else if (warp <= 2) {
        // ------------------------------------------------------------ products of one group
        const bool leader = tc::elect_one_sync();
        const int wg = warp - 1;
        const uint32_t idesc_x = tc::idesc_bf16(128, 128, false, false);         // X C^T
        const uint32_t idesc_s = tc::idesc_bf16(128, D, false, !GRAD);           // X S (S [inner][columns]) or X S^T
        const uint32_t idesc_r = tc::idesc_bf16(128, D, false, true);            // P R
        const uint32_t sm = tc::smem_u32(smem), t = tmem + wg * 256;
        const uint64_t dr = tc::sdesc(sm + L::kOffR, 16384, 1024);
        const uint64_t dx = tc::sdesc(sm + L::kOffX + wg * L::kTile, 16, 1024);
        bool r_seen = true;                      // this warp has waited for its pair's C, S and R
        auto wait_cs = [&](int pair) -> bool {
            return tc::warp_wait(&B.c_full, pair & 1, a.wait_err) && tc::warp_wait(&B.st_full, pair & 1, a.wait_err);
        };
        auto wait_r = [&](int pair) -> bool {
            r_seen = true;
            return tc::warp_wait(&B.r_full, pair & 1, a.wait_err) &&
                   tc::warp_wait(&B.r_ready[pair & 1], (pair >> 1) & 1, a.wait_err);
        };
        for (; more; more = w.next()) {
            if (w.first && w.pair > 0) {
                // This warp is through with the pair before (both warps say so of every pair, and both
                // see every pair arrive, so that no wait for a phase can fall a whole period behind).
                if (!r_seen && !(wait_cs(w.pair - 1) && wait_r(w.pair - 1))) break;
                if (leader) {
                    tc::mma_commit(&B.pair_empty);
                    tc::mma_commit(&B.r_empty);
                }
                __syncwarp();
            }
            if (w.first) r_seen = false;
            if ((w.it & 1) != wg) continue;
            const int n = w.it >> 1;             // heads of this group before
            if (!tc::warp_wait(&B.c_full, w.pair & 1, a.wait_err)) break;
            if (!tc::warp_wait(&B.x_full[wg], n & 1, a.wait_err)) break;
            tc::tc_fence_after();
            if (leader) {                        // (over the weights of the head before: its second product is ahead of this one)
                const uint64_t dc = tc::sdesc(sm, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
                    tc::mma_bf16(t, tc::sdesc_at(dx, at), tc::sdesc_at(dc, at), idesc_x, k > 0);
                }
                tc::mma_commit(&B.s_full[wg]);
            }
            __syncwarp();
            if (!tc::warp_wait(&B.st_full, w.pair & 1, a.wait_err)) break;
            if (n > 0 && !tc::warp_wait(&B.o_free[wg], (n - 1) & 1, a.wait_err)) break;
            tc::tc_fence_after();
            if (leader) {
                const uint64_t ds = GRAD ? tc::sdesc(sm + L::kOffS, 16, 1024) : tc::sdesc(sm + L::kOffS, D * 128, 1024);
#pragma unroll
                for (int k = 0; k < TERMS * D / 16; ++k) {       // the first terms' inner indices, then the second ones'
                    const int c = k % (D / 16), term = k / (D / 16) * L::kState;
                    tc::mma_bf16(t + 128, tc::sdesc_at(dx, (c >> 2) * 16384 + (c & 3) * 32),
                                 tc::sdesc_at(ds, term + (GRAD ? (c >> 2) * (D * 128) + (c & 3) * 32 : c * 2048)), idesc_s, k > 0);
                }
                tc::mma_commit(&B.o_full[wg]);   // X S': the output's first phase of a head
                tc::mma_commit(&B.x_empty[wg]);
            }
            __syncwarp();
            if (!r_seen && !wait_r(w.pair)) break;
            // (the weights of keys 64 .. are still being formed during the first half)
            if (!tc::warp_wait(&B.p_half[wg], n & 1, a.wait_err)) break;
            tc::tc_fence_after();
            if (leader)
#pragma unroll
                for (int k = 0; k < 4 * TERMS; ++k)
                    tc::mma_bf16_ts(t + 128, t + p_col(k & 3, k >> 2), tc::sdesc_at(dr, (k & 3) * 2048), idesc_r, 1u);
            __syncwarp();
            if (!tc::warp_wait(&B.p_full[wg], n & 1, a.wait_err)) break;
            tc::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int k = 0; k < 4 * TERMS; ++k)
                    tc::mma_bf16_ts(t + 128, t + p_col(4 + (k & 3), k >> 2), tc::sdesc_at(dr, (4 + (k & 3)) * 2048), idesc_r, 1u);
                tc::mma_commit(&B.o_full[wg]);   // the whole output: its second phase
            }
            __syncwarp();
        }
        if (leader) {                            // nothing of ours may still run on the tensor core at exit
            tc::mma_commit(&B.drain[wg]);
            tc::drain_wait(&B.drain[wg], 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ weights and outputs
        const int wg = (warp - 3) >> 2, quad = warp & 3, i = quad * 32 + lane;   // row of the chunk
        const int t128 = (threadIdx.x - 96) & 127;
        const uint32_t t = tmem + ((uint32_t)(quad * 32) << 16) + wg * 256;
        const float scale = rsqrtf((float)D);
        const LinRows& out = GRAD ? a.dq : a.o;
        uint8_t* stage = smem + L::kOffStage + (warp - 3) * L::kStage;
        // l's powers, kept while the KV head stays; each group has tables of its own:
        // l^(x - 31) for x >= 31, else 0, and l^(31 - x).
        __shared__ float diag[2][64];
        __shared__ __align__(16) float up[2][32];
        int h_of = -1;
        float rb[3], li1 = 0.f;
        bool ok = true;
        // A warp's box holds half of its columns. The other half's turn is behind the next head's
        // weights, when the first has long left (shared memory has no room for both).
        uint32_t o1[D / 4];
        int left1 = 0, head1 = 0, row1 = 0;
        auto put_second = [&]() {
            if (left1 <= 0) return;
            if (lane == 0) tc::bulk_wait_read();
            __syncwarp();
            store_half<D>(o1, &map_out, stage, lane, left1, D / 2, head1, row1, out);
            left1 = 0;
        };
        for (; more; more = w.next()) {
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
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.s_full[wg], (w.it >> 1) & 1, a.wait_err));
            if (ok && w.first) {
                if (w.c.rows < kL) {             // what lies behind the sequence may be anything
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.r_full, w.pair & 1, a.wait_err));
                    if (ok) zero_tail<D>(smem + L::kOffR, w.c.rows, t128, 128);
                    tc::fence_proxy_async_smem();
                }
                tc::mbar_arrive(&B.r_ready[w.pair & 1]);
            }
            if (!ok) continue;
            tc::tc_fence_after();
            // Blocks left of the diagonal's, then the diagonal's, then nothing.
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                uint32_t pk[16 * TERMS];         // first terms, second ones
                if (b > quad) {
#pragma unroll
                    for (int e = 0; e < 16 * TERMS; ++e) pk[e] = 0u;
                } else {
                    uint32_t r[32];
                    tc::tmem_ld32(t + 32 * b, r);
                    tc::tmem_wait_ld(r);
                    if (b < quad) {
                        const float f1 = b == 0 ? rb[0] : b == 1 ? rb[1] : rb[2];
                        const f32x2 f = pack2(f1, f1);
                        const ulonglong2* u = reinterpret_cast<const ulonglong2*>(up[wg]);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const ulonglong2 k = u[e / 2];
                            put_pair_terms<TERMS>(pk, e, mul2(pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), mul2(k.x, f)));
                            put_pair_terms<TERMS>(pk, e + 1, mul2(pack2(__uint_as_float(r[2 * e + 2]), __uint_as_float(r[2 * e + 3])), mul2(k.y, f)));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = 2 * e <= lane ? __uint_as_float(r[2 * e]) * diag[wg][lane - 2 * e + 31] : 0.f;
                            const float y = 2 * e + 1 <= lane ? __uint_as_float(r[2 * e + 1]) * diag[wg][lane - 2 * e + 30] : 0.f;
                            put_pair_terms<TERMS>(pk, e, pack2(x, y));
                        }
                    }
                }
                store_block<TERMS>(t + 32 * b, pk);
                if (b == 1) {                    // X S', scaled: the first half of the second product may start
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.o_full[wg], 0, a.wait_err));
                    if (!ok) break;
                    tc::tc_fence_after();
                    scale_half<D>(t + 128, li1);
                    scale_half<D>(t + 128 + D / 2, li1);
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&B.p_half[wg]);
                }
            }
            if (!ok) continue;
            tc::tmem_wait_st();
            tc::tc_fence_before();
            tc::mbar_arrive(&B.p_full[wg]);
            put_second();
            if (lane == 0) tc::bulk_wait_read();     // the last head's boxes have left the stage
            __syncwarp();
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.o_full[wg], 1, a.wait_err));
            if (!ok) continue;
            tc::tc_fence_after();
            // The rows leave tensor memory first: the next head's products need not wait for the stores.
            uint32_t o0[D / 4];
            load_half<D>(t + 128, scale, o0);
            load_half<D>(t + 128 + D / 2, scale, o1);
            tc::tc_fence_before();
            tc::mbar_arrive(&B.o_free[wg]);
            left1 = w.c.rows - 32 * quad;
            head1 = w.head;
            row1 = w.c.row0 + 32 * quad;
            store_half<D>(o0, &map_out, stage, lane, left1, 0, head1, row1, out);
        }
        put_second();
        if (lane == 0) bulk_wait();
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
    static constexpr uint32_t kOffG2 = kOffQ + kTile;                // G's second terms, then the second head's Q
    static constexpr uint32_t kSmem = kOffDo + 2 * kTile + 1024;
    static constexpr uint32_t kColDv = 256, kColDk = 256 + D;
};
constexpr int kColsThreads = 3 * 32 + 2 * 256;

struct ColsBarriers {
    uint64_t k_full, v_full, g_full, q_full[2], do_full[2], q_empty[2], do_empty[2];
    uint64_t q_ready[2], do_ready[2];            // their tails zeroed (a chunk of less than 128 rows)
    uint64_t s_full[2], init_full[2], p_half[2], p_full[2], acc_full[2];          // by group
    uint32_t tmem_base;
};

// dV = scale sum_heads ((Q K^T) o M)^T dO + diag(l^(m-1-j)) K G and dK = scale
// sum_heads ((dO V^T) o M)^T Q + diag(l^(m-1-j)) V G^T of one chunk and KV head.
// Scores are formed transposed (keys are the accumulator's rows): K Q^T in
// columns [0, 128) for one group of eight warps (dV), V dO^T in [128, 256) for
// another (dK), each with an issuing warp of its own; their weighted values' bf16 terms
// overwrite them as A operands, in two halves of the queries, so that the second product of
// one runs while the weights of the other are formed. dV and dK stay in tensor memory over all heads; they start as
// K G and V G^T, scaled there by l^(m-1-j) / scale. What bounds it is a head's chain of
// score product, weighting and second product, 2.6 us, in each of a unit's g heads: 4096 rows,
// 28/4 heads of d 128 (128 CTAs of seven heads) take 28 us, with one term 23.
template <int D, int TERMS>
__global__ void __launch_bounds__(kColsThreads, 1)
lin_cols_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                   const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_dv,
                   const __grid_constant__ CUtensorMap map_dk, const LinArgs a) {
    using L = ColsLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) ColsBarriers B;
    __shared__ float diag[64];
    __shared__ __align__(16) float pw[32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, f = blockIdx.x, h = blockIdx.y;
    LinChunk c;
    if (!lin_chunk<kL>(a, f, c)) {
        launch_dependents();
        wait_for_kernels();                      // a kernel never ends before the one it may overlap
        return;
    }
    const int g = a.Hq / a.Hkv;
    const bool tail = c.rows < kL;
    const float g2 = lin_g2(a, h);
    if (threadIdx.x < 64) diag[threadIdx.x] = threadIdx.x >= 31 ? lin_pow(g2, threadIdx.x - 31) : 0.f;
    else if (threadIdx.x < 96) pw[threadIdx.x - 64] = lin_pow(g2, threadIdx.x - 64);
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&B.q_full[s], 1);
            tc::mbar_init(&B.do_full[s], 1);
            tc::mbar_init(&B.q_empty[s], 2);
            tc::mbar_init(&B.do_empty[s], 2);
            tc::mbar_init(&B.q_ready[s], 256);
            tc::mbar_init(&B.do_ready[s], 256);
            tc::mbar_init(&B.s_full[s], 1);
            tc::mbar_init(&B.init_full[s], 1);
            tc::mbar_init(&B.p_half[s], 256);
            tc::mbar_init(&B.p_full[s], 256);
            tc::mbar_init(&B.acc_full[s], 1);
        }
        tc::mbar_init(&B.k_full, 1);
        tc::mbar_init(&B.v_full, 1);
        tc::mbar_init(&B.g_full, 1);
        tc::fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(&B.tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    // (only now: the next kernel could otherwise be given an SM's tensor memory before this
    // one, which waits for room there, and then wait for this one)
    launch_dependents();
    const uint32_t tmem = B.tmem_base;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        const int row = (int)c.row0;
        int n = 0;
        for (int i = 0; i < g; ++i) {
            const int s = i & 1;
            if (TERMS == 2 && i == 1)            // the second head's Q takes the place of G's second terms
                if (!tc::warp_wait(&B.init_full[0], 0, a.wait_err) || !tc::warp_wait(&B.init_full[1], 0, a.wait_err)) break;
            if (i >= 2 && !tc::warp_wait(&B.q_empty[s], ((i >> 1) - 1) & 1, a.wait_err)) break;
            if (i >= 2 && !tc::warp_wait(&B.do_empty[s], ((i >> 1) - 1) & 1, a.wait_err)) break;
            if (lane == 0) {
                if (i == 0) {
                    tc::mbar_arrive_expect_tx(&B.k_full, L::kTile);
                    tc::mbar_arrive_expect_tx(&B.v_full, L::kTile);
                }
                tc::mbar_arrive_expect_tx(&B.q_full[s], L::kTile);
                tc::mbar_arrive_expect_tx(&B.do_full[s], L::kTile);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    if (i == 0) tc::tma_load_3d(smem + b * 16384, &map_k, &B.k_full, 64 * b, h, row);
                    tc::tma_load_3d(smem + L::kOffQ + s * L::kTile + b * 16384, &map_q, &B.q_full[s], 64 * b, h * g + i, row);
                }
#pragma unroll
                for (int b = 0; b < D / 64; ++b) {
                    if (i == 0) tc::tma_load_3d(smem + L::kOffV + b * 16384, &map_v, &B.v_full, 64 * b, h, row);
                    tc::tma_load_3d(smem + L::kOffDo + s * L::kTile + b * 16384, &map_do, &B.do_full[s], 64 * b, h * g + i, row);
                }
            }
            n = i + 1;
            if (i == 0) {
                wait_for_kernels();              // the gradients of the states
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&B.g_full, TERMS * L::kState);
#pragma unroll
                    for (int b = 0; b < D / 64; ++b) {
                        tc::tma_load_2d(smem + L::kOffG + b * (D * 128), &map_g, &B.g_full, 64 * b, (f * a.Hkv + h) * D);
                        if (TERMS == 2) tc::tma_load_2d(smem + L::kOffG2 + b * (D * 128), &map_g, &B.g_full, D + 64 * b, (f * a.Hkv + h) * D);
                    }
                }
            }
        }
        // None of this CTA's copies may still be landing when it exits.
        if (lane == 0) {
            tc::drain_wait(&B.k_full, 0);
            tc::drain_wait(&B.v_full, 0);
            tc::drain_wait(&B.g_full, 0);
            for (int i = max(0, n - 2); i < n; ++i) {
                tc::drain_wait(&B.q_full[i & 1], (i >> 1) & 1);
                tc::drain_wait(&B.do_full[i & 1], (i >> 1) & 1);
            }
        }
    } else if (warp <= 2) {
        // ------------------------------------------------------------ products: dV's (x 0), dK's (x 1)
        const bool leader = tc::elect_one_sync();
        const int x = warp - 1;
        const uint32_t id_s = tc::idesc_bf16(128, 128, false, false), id_acc = tc::idesc_bf16(128, D, false, true);
        const uint32_t id_g = tc::idesc_bf16(128, D, false, x == 0);
        const uint32_t sm = tc::smem_u32(smem), t = tmem + 128 * x, acc = tmem + (x ? L::kColDk : L::kColDv);
        const uint64_t dc = tc::sdesc(sm + (x ? L::kOffV : 0), 16, 1024);        // keys' operand
        const uint32_t own = x ? L::kOffDo : L::kOffQ, other = x ? L::kOffQ : L::kOffDo;     // scores' operand, the product's
        uint64_t* own_full = tail ? (x ? B.do_ready : B.q_ready) : (x ? B.do_full : B.q_full);
        uint64_t* other_full = tail ? (x ? B.q_ready : B.do_ready) : (x ? B.q_full : B.do_full);
        uint64_t *own_empty = x ? B.do_empty : B.q_empty, *other_empty = x ? B.q_empty : B.do_empty;
        bool ok = tc::warp_wait(x ? &B.v_full : &B.k_full, 0, a.wait_err);
        for (int i = 0; ok && i < g; ++i) {
            const int s = i & 1;
            if (!tc::warp_wait(&own_full[s], (i >> 1) & 1, a.wait_err)) break;
            tc::tc_fence_after();
            if (leader) {
                const uint64_t db = tc::sdesc(sm + own + s * L::kTile, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
                    tc::mma_bf16(t, tc::sdesc_at(dc, at), tc::sdesc_at(db, at), id_s, k > 0);
                }
                tc::mma_commit(&B.s_full[x]);
                tc::mma_commit(&own_empty[s]);
            }
            __syncwarp();
            if (i == 0) {
                if (!tc::warp_wait(&B.g_full, 0, a.wait_err)) break;
                tc::tc_fence_after();
                if (leader) {
                    const uint64_t dg = x ? tc::sdesc(sm + L::kOffG, 16, 1024) : tc::sdesc(sm + L::kOffG, D * 128, 1024);
#pragma unroll
                    for (int k = 0; k < TERMS * D / 16; ++k) {   // the first terms' inner indices, then the second ones'
                        const int c = k % (D / 16), term = k / (D / 16) * (L::kOffG2 - L::kOffG);
                        tc::mma_bf16(acc, tc::sdesc_at(dc, (c >> 2) * 16384 + (c & 3) * 32),
                                     tc::sdesc_at(dg, term + (x ? (c >> 2) * (D * 128) + (c & 3) * 32 : c * 2048)), id_g, k > 0);
                    }
                    tc::mma_commit(&B.init_full[x]);
                }
                __syncwarp();
            }
            // (the weights of the other blocks of queries are still being formed during the first half)
            if (!tc::warp_wait(&B.p_half[x], i & 1, a.wait_err)) break;
            if (!tc::warp_wait(&other_full[s], (i >> 1) & 1, a.wait_err)) break;
            tc::tc_fence_after();
            const uint64_t db = tc::sdesc(sm + other + s * L::kTile, 16384, 1024);
            auto product = [&](int first) {      // blocks first, first + 2
#pragma unroll
                for (int n = 0; n < 4 * TERMS; ++n) {
                    const int k = 2 * first + (n & 2) * 2 + (n & 1);
                    tc::mma_bf16_ts(acc, t + p_col(k, n >> 2), tc::sdesc_at(db, k * 2048), id_acc, 1u);
                }
            };
            if (leader) product(0);
            __syncwarp();
            if (!tc::warp_wait(&B.p_full[x], i & 1, a.wait_err)) break;
            tc::tc_fence_after();
            if (leader) {
                product(1);
                tc::mma_commit(&other_empty[s]);
            }
            __syncwarp();
        }
        if (leader) {                            // (also: nothing of ours may still run on the tensor core at exit)
            tc::mma_commit(&B.acc_full[x]);
            tc::drain_wait(&B.acc_full[x], 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ weights and outputs
        const int x = (warp - 3) >> 3, half = (warp - 3) >> 2 & 1, quad = warp & 3, j = quad * 32 + lane;      // key row of the chunk
        const int t256 = (threadIdx.x - 96) & 255;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), t = lanes + 128 * x;
        const uint32_t acc = lanes + (x ? L::kColDk : L::kColDv) + D / 2 * half;
        const float scale = rsqrtf((float)D);
        // A chunk's tail: group 0 zeroes Q's rows, group 1 dO's.
        auto tails = [&](int i) -> bool {
            const int s = i & 1;
            uint64_t* full = x ? B.do_full : B.q_full;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], (i >> 1) & 1, a.wait_err))) return false;
            zero_tail<D>(smem + (x ? L::kOffDo : L::kOffQ) + s * L::kTile, c.rows, t256, 256);
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(x ? &B.do_ready[s] : &B.q_ready[s]);
            return true;
        };
        float rb[2];                             // of blocks 2 half, 2 half + 1
#pragma unroll
        for (int b = 0; b < 2; ++b) rb[b] = 2 * half + b > quad ? lin_pow(g2, 32 * (2 * half + b) - j) : 0.f;
        bool ok = !tail || tails(0);
        for (int i = 0; ok && i < g; ++i) {
            if (tail && i > 0 && i + 1 < g && !(ok = tails(i + 1))) break;
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.s_full[x], i & 1, a.wait_err));
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int block = 2 * half + b;  // queries 32 block ..
                uint32_t pk[16 * TERMS];         // first terms, second ones
                uint32_t r[32];
                if (block >= quad) {
                    tc::tmem_ld32(t + 32 * block, r);
                    tc::tmem_wait_ld(r);
                    const int left = c.rows - 32 * block;
                    if (left < 32) {             // queries behind the sequence: anything
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = e < left ? r[e] : 0u;
                    }
                }
                if (block < quad) {
#pragma unroll
                    for (int e = 0; e < 16 * TERMS; ++e) pk[e] = 0u;
                } else if (block > quad) {
                    const f32x2 f = pack2(rb[b], rb[b]);
                    const ulonglong2* u = reinterpret_cast<const ulonglong2*>(pw);
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const ulonglong2 k = u[e / 2];
                        put_pair_terms<TERMS>(pk, e, mul2(pack2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), mul2(k.x, f)));
                        put_pair_terms<TERMS>(pk, e + 1, mul2(pack2(__uint_as_float(r[2 * e + 2]), __uint_as_float(r[2 * e + 3])), mul2(k.y, f)));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float p0 = 2 * e >= lane ? __uint_as_float(r[2 * e]) * diag[2 * e - lane + 31] : 0.f;
                        const float p1 = 2 * e + 1 >= lane ? __uint_as_float(r[2 * e + 1]) * diag[2 * e + 32 - lane] : 0.f;
                        put_pair_terms<TERMS>(pk, e, pack2(p0, p1));
                    }
                }
                store_block<TERMS>(t + 32 * block, pk);
                if (b == 0 && i == 0) continue;  // (the first head's products wait for G: all weights first)
                if (i == 0) {
                    ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.init_full[x], 0, a.wait_err));
                    if (!ok) break;
                    tc::tc_fence_after();
                    scale_half<D>(acc, j < c.rows ? lin_pow(g2, c.rows - 1 - j) / scale : 0.f);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                if (b == 0 || i == 0) tc::mbar_arrive(&B.p_half[x]);
                if (b == 1) tc::mbar_arrive(&B.p_full[x]);
            }
            if (!ok) break;
            if (tail && i == 0 && g > 1) ok = tails(1);      // (behind the products with G, whose place Q's second tile takes)
        }
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.acc_full[x], 0, a.wait_err));
        if (ok) {
            tc::tc_fence_after();
            uint32_t o[D / 4];
            load_half<D>(acc, scale, o);
            // (staged where K lay for group 0, V for group 1: no other product has read them)
            store_half<D>(o, x ? &map_dk : &map_dv, smem + (x ? L::kOffV : 0) + ((warp - 3) & 7) * (32 * D), lane, c.rows - 32 * quad,
                          D / 2 * half, h, c.row0 + 32 * quad, x ? a.dk : a.dv);
        }
        if (lane == 0) bulk_wait();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ launches

bool rows_map(CUtensorMap* m, const LinRows& x, int H, const LinArgs& a, int rows, std::string* why) {
    return make_tmap_3d(m, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.d, H, a.n, a.d * 2, x.stride * 2, 64, 1, rows, why);
}
// Of an output, as store_half writes it.
bool half_map(CUtensorMap* m, const LinRows& x, int H, const LinArgs& a, std::string* why) {
    return make_tmap_3d(m, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.d, H, a.n, a.d * 2, x.stride * 2, a.d / 2, 1, 32, why,
                        a.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}
bool sums_map(CUtensorMap* m, const float* p, const LinArgs& a, std::string* why) {
    return make_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.d, (uint64_t)a.n_chunks * a.Hkv * a.d, a.d * 4, 32, 32, why);
}
// The states as the scan leaves them: rows of d first and d second terms.
bool states_map(CUtensorMap* m, const float* p, const LinArgs& a, std::string* why) {
    return make_tmap_2d(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2 * a.d, (uint64_t)a.n_chunks * a.Hkv * a.d, a.d * 4, 64, a.d, why);
}

// Launches a kernel that may start before the stream's last kernel, one of this
// file's, has ended; it waits for that one itself (wait_for_kernels) before it
// touches what that one writes. Each asks for the largest split of an SM's memory in
// favour of shared memory, as the tensor-core kernels need it: the scan, which needs
// none, otherwise had the split changed before and after it (4 us until the next
// kernel started).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
    cfg.gridDim = grid; cfg.blockDim = dim3(threads); cfg.dynamicSmemBytes = smem; cfg.stream = s;
    cfg.attrs = attr; cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The chunks' sums and their scans: k v^T, in a backward (BOTH) also q do^T. The
// forward's sums kernel is held to registers that leave room for the scan's CTAs beside
// it, so that their set-up overlaps (4096 rows, 4 KV heads of d 128: 1.7 us of 31); the
// backward's is much longer and faster with more (0.64 us a stage instead of 0.75).
template <int D, int TERMS, bool BOTH> cudaError_t states(const LinArgs& a, cudaStream_t s, std::string* why) {
    static SmemGrant grant;
    cudaError_t e = allow_smem(lin_part_tc_kernel<D, BOTH>, PartLayout<D>::kSmem, grant);
    if (e != cudaSuccess) return e;
    const int nz = BOTH ? 2 : 1;
    if (a.n) {
        CUtensorMap k, v, q, go, out, gout;
        if (!rows_map(&k, a.k, a.Hkv, a, kPartRows, why) || !rows_map(&v, a.v, a.Hkv, a, kPartRows, why) || !sums_map(&out, a.part, a, why))
            return cudaErrorInvalidValue;
        q = k; go = v; gout = out;               // (unused by a forward)
        if (BOTH && (!rows_map(&q, a.q, a.Hq, a, kPartRows, why) || !rows_map(&go, a.dout, a.Hq, a, kPartRows, why) ||
                     !sums_map(&gout, a.gpart, a, why)))
            return cudaErrorInvalidValue;
        const int grid = std::min(a.n_chunks * a.Hkv * nz, sm_count());
        ProfScope ps("lin_part_tc_kernel", s);
        lin_part_tc_kernel<D, BOTH><<<grid, kPartThreads, PartLayout<D>::kSmem, s>>>(q, k, v, go, out, gout, a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)(a.n_seq * a.Hkv * (D * D / 4 / kScanThreads)), nz);
    ProfScope ps("lin_scan_bf16_kernel", s);
    if (a.n) return launch_after(lin_scan_bf16_kernel<D, TERMS>, grid, kScanThreads, 0, s, a);
    lin_scan_bf16_kernel<D, TERMS><<<grid, kScanThreads, 0, s>>>(a);                    // no sums before it
    return cudaGetLastError();
}

template <int D, int TERMS, bool GRAD> cudaError_t rows(const LinArgs& a, cudaStream_t s, std::string* why) {
    static SmemGrant grant;
    const cudaError_t e = allow_smem(lin_rows_tc_kernel<D, GRAD, TERMS>, RowsLayout<D, TERMS>::kSmem, grant);
    if (e != cudaSuccess) return e;
    CUtensorMap x, c, r, st, out;
    if (!rows_map(&x, GRAD ? a.dout : a.q, a.Hq, a, kL, why) || !rows_map(&c, GRAD ? a.v : a.k, a.Hkv, a, kL, why) ||
        !rows_map(&r, GRAD ? a.k : a.v, a.Hkv, a, kL, why) || !states_map(&st, a.part, a, why) ||
        !half_map(&out, GRAD ? a.dq : a.o, a.Hq, a, why))
        return cudaErrorInvalidValue;
    const int heads = a.n_chunks * a.Hq, units = a.n_chunks * a.Hkv, grid = std::min(heads, sm_count());
    ProfScope ps("lin_rows_tc_kernel", s);
    return launch_after(lin_rows_tc_kernel<D, GRAD, TERMS>, dim3(grid), kRowsThreads, RowsLayout<D, TERMS>::kSmem, s, x, c, r, st,
                        out, a, Cut{heads / grid, heads % grid, units >= 8 * grid ? units : 0});
}

template <int D, int TERMS> cudaError_t cols(const LinArgs& a, cudaStream_t s, std::string* why) {
    static SmemGrant grant;
    const cudaError_t e = allow_smem(lin_cols_tc_kernel<D, TERMS>, ColsLayout<D>::kSmem, grant);
    if (e != cudaSuccess) return e;
    CUtensorMap q, k, v, go, gs, dv, dk;
    if (!rows_map(&q, a.q, a.Hq, a, kL, why) || !rows_map(&k, a.k, a.Hkv, a, kL, why) || !rows_map(&v, a.v, a.Hkv, a, kL, why) ||
        !rows_map(&go, a.dout, a.Hq, a, kL, why) || !states_map(&gs, a.gpart, a, why) ||
        !half_map(&dv, a.dv, a.Hkv, a, why) || !half_map(&dk, a.dk, a.Hkv, a, why))
        return cudaErrorInvalidValue;
    ProfScope ps("lin_cols_tc_kernel", s);
    return launch_after(lin_cols_tc_kernel<D, TERMS>, dim3(a.n_chunks, a.Hkv), kColsThreads, ColsLayout<D>::kSmem, s, q, k, v, go, gs, dv,
                        dk, a);
}

template <int D, int TERMS> cudaError_t fwd(const LinArgs& a, cudaStream_t s, std::string* why) {
    const cudaError_t e = states<D, TERMS, false>(a, s, why);
    return e != cudaSuccess || !a.n ? e : rows<D, TERMS, false>(a, s, why);
}

template <int D, int TERMS> cudaError_t bwd(const LinArgs& a, cudaStream_t s, std::string* why) {
    cudaError_t e = states<D, TERMS, true>(a, s, why);
    if (e == cudaSuccess && a.n) e = cols<D, TERMS>(a, s, why);
    return e != cudaSuccess || !a.n ? e : rows<D, TERMS, true>(a, s, why);
}

}  // namespace

cudaError_t launch_lin_fwd_tc(const LinArgs& a, cudaStream_t s, std::string* why) {
    if (a.one_term) return a.d == 128 ? fwd<128, 1>(a, s, why) : fwd<64, 1>(a, s, why);
    return a.d == 128 ? fwd<128, 2>(a, s, why) : fwd<64, 2>(a, s, why);
}

cudaError_t launch_lin_bwd_tc(const LinArgs& a, cudaStream_t s, std::string* why) {
    if (a.one_term) return a.d == 128 ? bwd<128, 1>(a, s, why) : bwd<64, 1>(a, s, why);
    return a.d == 128 ? bwd<128, 2>(a, s, why) : bwd<64, 2>(a, s, why);
}

}  // namespace pkv
