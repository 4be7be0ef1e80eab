// Attention of a few queries (one generated token, a handful of drafted ones)
// against a long paged cache, bf16, with modified scores (mod.cuh).
//
// Bound by reading K and V once: 2 * keys * Hkv * d * 2 bytes. The rows of a
// 16-row tile are (query, head) pairs of one KV group, so a group's heads share
// each key. A CTA owns (KV head, row tile, share of the keys); its 8 warps take
// 16 keys each of every 128, with online softmax states of their own that meet
// in shared memory at the end. Shares of the keys meet in attn_join.
//
// A page's rows of one KV head are contiguous, so a producer warp streams K and
// V by untiled bulk copies into a ring of steps of 128 keys (192 KB of it: HBM's
// latency and rate ask for 45 KB in flight per SM). One token on 131072 keys, 28/4
// heads, d 128: 44 us for 268 MB, 6.1 TB/s, 0.90 of the measured rate, and 6 us for
// the join. The rows keep their order, without padding: K's 16-byte reads meet two to
// a bank, V's four, 1500 cycles of the 2700 that a step's bytes take to arrive.
//
// The 16x8x16 bf16 MMA takes its operands from 16-byte reads because the order
// of the products' inner index is free:
//   S = Q K^T   lane (n = lane / 4, t = lane % 4) holds dims 8t .. 8t + 7 of a
//               32-dim block of key n: two k-steps' worth of its B operand, if
//               Q's fragments take the same dims;
//   O += P V    lane (g = lane / 4, t) holds dims 8g .. 8g + 7 of a 64-dim block
//               of keys 2t, 2t + 1, 2t + 8, 2t + 9: the B operands of the 8
//               products whose column v stands for dim 8v + j, j = 0 .. 7, after
//               pairing neighbouring keys' halves with byte permutes.
// The tensor core idles mostly (16 rows), so the legacy MMA serves: tensor memory
// would only add steps.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mod.cuh"
#include "tc.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8, kThreads = 32 * (kWarps + 1);   // and the producer warp
constexpr int kRows = 16, kKeys = 16;                 // rows of a tile, keys of a warp's block
constexpr int kStep = kWarps * kKeys;                 // keys of a CTA's step

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D> struct Ring {
    static constexpr int kTile = kStep * D * 2;               // K or V of a step, bytes
    static constexpr int kStages = 96 * 1024 / kTile;         // 3 (d 128) or 6 (d 64)
    static constexpr int kBytes = 2 * kStages * kTile;
    static_assert(kBytes >= kWarps * kRows * (D + 4) * 4, "the warps' results fit the ring");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(AttnArgs a) {
    using R = Ring<D>;
    extern __shared__ __align__(128) uint8_t ring[];  // stages of K, V; then [kWarps][kRows][D + 4] floats
    float* part = reinterpret_cast<float*>(ring);
    __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
    __shared__ uint64_t full[R::kStages], empty[R::kStages];
    __shared__ uint32_t good[R::kStages];             // bit w: the stage holds the keys of warp w's block
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int kvh = blockIdx.y, group = a.Hq / a.Hkv;
    const int row0 = (int)blockIdx.x * kRows, rows = (int)min64(kRows, a.n_q * group - row0);
    // Lane's rows g and g + 8: visible keys, position, slope. Rows past the end see nothing.
    int2 range[2];
    int pos[2];
    float slope2[2];
    int lo = 0x7fffffff, hi = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = min(g + 8 * u, rows - 1), i = (row0 + r) / group;
        range[u] = g + 8 * u < rows ? row_range(a.m, a.q_start, i) : make_int2(0, 0);
        pos[u] = (int)a.q_start + i;
        slope2[u] = a.m.slopes ? a.m.slopes[kvh * group + (row0 + r) % group] * kLog2e : 0.f;
        if (range[u].y > 0) {
            lo = min(lo, range[u].x);
            hi = max(hi, range[u].y);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    // This CTA's steps of 128 keys.
    const int s0 = hi > 0 ? lo / kStep : 0, n = hi > 0 ? (hi + kStep - 1) / kStep - s0 : 0;
    const int b0 = s0 + (int)((int64_t)n * blockIdx.z / gridDim.z), b1 = s0 + (int)((int64_t)n * (blockIdx.z + 1) / gridDim.z);
    const int end = min(hi, b1 * kStep);
    // The join of the shares may take its place beside these CTAs (it waits for their end).
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int st = 0; st < R::kStages; ++st) {
            tc::mbar_init(&full[st], 1);
            tc::mbar_init(&empty[st], kWarps);
        }
        tc::fence_barrier_init();
    }
    __syncthreads();

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        int issued = b0;
        for (int b = b0; b < b1; ++b) {
            const int st = (b - b0) % R::kStages, turn = (b - b0) / R::kStages;
            if (turn > 0 && !tc::warp_wait(&empty[st], (turn - 1) & 1, a.err)) break;
            // The step's keys in runs that lie in one page, up to a whole block past `end`
            // (pages are whole blocks): lane l looks up the l-th run's page.
            const int k0 = b * kStep, k1 = min(k0 + kStep, (end + kKeys - 1) / kKeys * kKeys);
            const int first = k0 / a.P, runs = (k1 - 1) / a.P - first + 1;       // at most 9 (pages of 16)
            int32_t pp = -1;
            if (lane < runs) pp = a.bt[first + lane];
            const int from = max(k0, (first + lane) * a.P), to = min(k1, (first + lane + 1) * a.P);
            const bool ok = lane < runs && pp >= 0 && pp < a.num_phys;
            uint32_t blocks = (1u << kWarps) - 1, rows_in = (uint32_t)(k1 - k0);
            if (!__all_sync(0xffffffffu, ok || lane >= runs)) {
                // Runs without a usable page are left out: fine where no row sees their keys.
                for (uint32_t bad = __ballot_sync(0xffffffffu, lane < runs && !ok); bad; bad &= bad - 1) {
                    const int l = __ffs(bad) - 1;
                    const int f = __shfl_sync(0xffffffffu, from, l), e = __shfl_sync(0xffffffffu, to, l);
                    if (__any_sync(0xffffffffu, (range[0].x < e && range[0].y > f) || (range[1].x < e && range[1].y > f)) &&
                        lane == 0)
                        report_error(a.err, kErrBadPage);
                }
                // (Runs begin and end at blocks: pages are whole blocks.)
                blocks = __reduce_or_sync(0xffffffffu,
                                          ok ? (2u << ((to - k0 - 1) / kKeys)) - (1u << ((from - k0) / kKeys)) : 0u);
                rows_in = __reduce_add_sync(0xffffffffu, ok ? (uint32_t)(to - from) : 0u);
            }
            if (lane == 0) {
                good[st] = blocks;
                if (rows_in) tc::mbar_arrive_expect_tx(&full[st], 2u * rows_in * D * 2);
                else tc::mbar_arrive(&full[st]);
            }
            __syncwarp();
            if (ok) {
                const size_t src = (((size_t)pp * a.Hkv + kvh) * a.P + from % a.P) * D;
                uint8_t* dst = ring + 2 * st * R::kTile + (from - k0) * D * 2;
                const uint32_t bytes = (uint32_t)(to - from) * D * 2;
                tc::bulk_load(dst, static_cast<const __nv_bfloat16*>(a.kpool) + src, bytes, &full[st]);
                tc::bulk_load(dst + R::kTile, static_cast<const __nv_bfloat16*>(a.vpool) + src, bytes, &full[st]);
            }
            issued = b + 1;
        }
        // None of this CTA's copies may still be landing when it goes on.
        for (int b = max(b0, issued - R::kStages); b < issued; ++b)
            tc::drain_wait(&full[(b - b0) % R::kStages], ((b - b0) / R::kStages) & 1);
    }
    // ---------------------------------------------------------------- consumers
    uint32_t q[D / 16][4];
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (g + 8 * u < rows) {
                const int r = row0 + g + 8 * u;
                w = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                         ((size_t)(r / group) * a.Hq + kvh * group + r % group) * D) +
                          c * 4 + t);
            }
            // Words 2 s, 2 s + 1 belong to k-step s: its lower and upper 8 inner indices.
            q[2 * c][u] = w.x;
            q[2 * c][u + 2] = w.y;
            q[2 * c + 1][u] = w.z;
            q[2 * c + 1][u + 2] = w.w;
        }

    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    const float sl2 = rsqrtf((float)D) * kLog2e;

    auto compute = [&](int key0, const uint4* ks, const uint4* vs) {
        float s[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint4 k = ks[(8 * nt + g) * (D / 8) + c * 4 + t];
                mma16816(s[nt], q[2 * c], k.x, k.y);
                mma16816(s[nt], q[2 * c + 1], k.z, k.w);
            }
        }
        // Element e of tile nt: row g + 8 (e >> 1), key key0 + 8 nt + 2 t + (e & 1).
        if (a.m.cap > 0.f) {
            float top = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(s[e >> 2][e & 3]));
            if (warp_top(top) * a.m.k <= kTanhLong) {
                const f32x2 k2 = pack2(a.m.k, a.m.k), c2 = pack2(a.m.c2, a.m.c2);
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    unpack2(mul2(tanh_long2(mul2(pack2(s[e >> 2][e & 3], s[e >> 2][(e & 3) + 1]), k2)), c2),
                            s[e >> 2][e & 3], s[e >> 2][(e & 3) + 1]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] = a.m.c2 * tanh_any(s[e >> 2][e & 3] * a.m.k);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] *= sl2;
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int u = (e & 3) >> 1, key = key0 + 8 * (e >> 2) + 2 * t + (e & 1);
            float& z = s[e >> 2][e & 3];
            if (a.m.slopes) z = fmaf(-slope2[u], fabsf((float)(key - pos[u])), z);
            if (key < range[u].x || key >= range[u].y) z = -INFINITY;
            mx[u] = fmaxf(mx[u], z);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float mn = fmaxf(m[u], mx[u]);
                const float f = m[u] == -INFINITY ? 0.f : fast_exp2(m[u] - mn);
                m[u] = mn;
                l[u] *= f;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[j][2 * u] *= f;
                    o[j][2 * u + 1] *= f;
                }
            }
        }
        uint32_t pw[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // (A row that has seen nothing yet keeps m = -inf; its weights are 0.)
                const float ref = m[u] == -INFINITY ? 0.f : m[u];
                const float p0 = fast_exp2(s[nt][2 * u] - ref), p1 = fast_exp2(s[nt][2 * u + 1] - ref);
                l[u] += p0 + p1;                      // lane's own keys; the four lanes meet at the end
                pw[2 * nt + u] = pack_bf16x2(p0, p1); // P rounded to bf16 for the product, l from the unrounded
            }
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint4 v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = vs[(2 * t + (r & 1) + 8 * (r >> 1)) * (D / 8) + c * 8 + g];
            const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&v[0]);
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&v[1]);
            const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&v[2]);
            const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&v[3]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = j & 1 ? 0x7632 : 0x5410;          // high or low halves of two keys
                mma16816(o[8 * c + j], pw, __byte_perm(w0[j >> 1], w1[j >> 1], sel),
                         __byte_perm(w2[j >> 1], w3[j >> 1], sel));
            }
        }
    };
    if (warp < kWarps) {
        bool ok = true;
        for (int b = b0; ok && b < b1; ++b) {
            const int st = (b - b0) % R::kStages;
            ok = tc::warp_wait(&full[st], ((b - b0) / R::kStages) & 1, a.err);
            const int key0 = b * kStep + warp * kKeys;
            if (ok && (good[st] >> warp & 1) && key0 < end) {
                const uint8_t* base = ring + 2 * st * R::kTile + warp * kKeys * D * 2;
                compute(key0, reinterpret_cast<const uint4*>(base), reinterpret_cast<const uint4*>(base + R::kTile));
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[st]);
        }
    }
    __syncthreads();                                  // the ring is free

    // The warps' states meet: row r's maximum, sum and O.
    if (warp < kWarps)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (t == 0) {
            wm[warp][g + 8 * u] = m[u];
            wl[warp][g + 8 * u] = l[u];
        }
        float* dst = part + (warp * kRows + g + 8 * u) * (D + 4);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)               // columns v = 2t + h: dims 64 c + 8 v + j
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    *reinterpret_cast<float4*>(dst + 64 * c + 16 * t + 8 * h + j) =
                        make_float4(o[8 * c + j][2 * u + h], o[8 * c + j + 1][2 * u + h], o[8 * c + j + 2][2 * u + h],
                                    o[8 * c + j + 3][2 * u + h]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float top = wm[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, wm[w][r]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(wm[w][r] - ref);
            sum = fmaf(f, wl[w][r], sum);
            const float4 z = *reinterpret_cast<const float4*>(part + (w * kRows + r) * (D + 4) + c);
            acc.x = fmaf(f, z.x, acc.x); acc.y = fmaf(f, z.y, acc.y);
            acc.z = fmaf(f, z.z, acc.z); acc.w = fmaf(f, z.w, acc.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse2 = sum == 0.f ? -INFINITY : ref + log2f(sum);
        const int row = row0 + r, h = kvh * group + row % group;
        const size_t hrow = (size_t)h * a.n_q + row / group;
        if (a.splits > 1) {
            const size_t prow = (size_t)blockIdx.z * a.Hq * a.n_q + hrow;
            *reinterpret_cast<float4*>(a.part + prow * D + c) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (c == 0) a.part[(size_t)a.splits * a.Hq * a.n_q * D + prow] = lse2;
        } else {
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + ((size_t)(row / group) * a.Hq + h) * D + c) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (c == 0) a.lse[hrow] = lse2 * kLn2;
        }
    }
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    constexpr int smem = Ring<D>::kBytes;
    static SmemGrant allowed;
    const cudaError_t e = allow_smem(few_kernel<D>, smem, allowed);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)((a.n_q * (a.Hq / a.Hkv) + kRows - 1) / kRows);
    ProfScope ps("few_kernel", s);
    few_kernel<D><<<dim3(tiles, a.Hkv, a.splits), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Up to 16 queries: their 16-row tiles read each key ceil(n_q g / 16) times (from
// L2 but for the first), the tensor-core kernel's 128-row tiles once per head. Both
// sides on 131072 keys, this kernel and the tensor-core one, us (cap 50):
//              n_q = 8       16         24
//   28/4 d 128  138  257   237  259   384  257
//   64/8 d 64   204  507   400  507   789  508
//   8/8 d 128    87  142    90  142   139  142
//   32/2 d 128  138  259   292  257   384  257   (groups of 16 cross over at 14)
bool few_supported(const AttnArgs& a) {
    return a.dtype == PKV_BF16 && !a.sel && a.n_q <= 16 && a.P % kKeys == 0;
}

int attn_few_splits(const AttnArgs& a) {
    // One wave of CTAs, each with a step of 128 keys at least; up to 4 steps are
    // not worth a second kernel.
    const int sms = sm_count();
    const int64_t ctas = (a.n_q * (a.Hq / a.Hkv) + kRows - 1) / kRows * a.Hkv, steps = (a.m.n_keys + kStep - 1) / kStep;
    const int64_t room = std::max<int64_t>(1, sms / ctas);
    return steps <= 4 ? 1 : (int)std::min<int64_t>({steps, room, 512});
}

cudaError_t launch_attn_few(const AttnArgs& a, cudaStream_t s) {
    return a.d == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace pkv
