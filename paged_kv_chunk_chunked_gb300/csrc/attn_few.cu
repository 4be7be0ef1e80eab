// Attention of a few queries (one generated token, a handful of drafted ones)
// against a long paged cache, bf16, with modified scores (mod.cuh).
//
// Bound by reading K and V once: 2 * keys * Hkv * d * 2 bytes. The rows of a
// 16-row tile are (query, head) pairs of one KV group, so a group's heads share
// each key. A CTA owns (KV head, row tile, share of the keys); its 8 warps take
// 16 keys each of every 128, with online softmax states of their own that meet
// in shared memory at the end. Shares of the keys meet in attn_join.
//
// K and V go from global memory straight to the operand registers of the
// 16x8x16 bf16 MMA, 16 bytes per load, with no shared memory in between. That
// works because the order of the products' inner index is free:
//   S = Q K^T   lane (n = lane / 4, t = lane % 4) holds dims 8t .. 8t + 7 of a
//               32-dim block of key n: two k-steps' worth of its B operand, if
//               Q's fragments take the same dims;
//   O += P V    lane (g = lane / 4, t) holds dims 8g .. 8g + 7 of a 64-dim block
//               of keys 2t, 2t + 1, 2t + 8, 2t + 9: the B operands of the 8
//               products whose column v stands for dim 8v + j, j = 0 .. 7, after
//               pairing neighbouring keys' halves with byte permutes.
// The tensor core idles mostly (16 rows), so the legacy MMA serves: operands in
// tensor or shared memory would only add steps. The next 16 keys' 16 loads are
// in flight while a block is computed: 8 KB per warp, 64 KB per SM, above the
// 45 KB that HBM's latency and rate ask for per SM.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mod.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 16, kKeys = 16;                 // rows of a tile, keys of a warp's block
constexpr int kStep = kWarps * kKeys;                 // keys of a CTA's step

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A warp's 16 keys: K of keys lane / 4 and 8 + lane / 4, V of keys 2t, 2t + 1,
// 2t + 8, 2t + 9.
template <int D> struct Block {
    uint4 k[2][D / 32];
    uint4 v[4][D / 64];
    int key0;                                         // first key, or -1: no keys (past the share, or a bad page)
};

template <int D>
__device__ __forceinline__ void load_block(Block<D>& b, const AttnArgs& a, int key0, int end, int32_t pp, int kvh, int lane) {
    b.key0 = -1;
    if (key0 >= end) return;
    if (pp < 0 || pp >= a.num_phys) {
        if (lane == 0) report_error(a.err, kErrBadPage);
        return;
    }
    b.key0 = key0;
    const size_t base = (((size_t)pp * a.Hkv + kvh) * a.P + key0 % a.P) * D;
    const uint4* kp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.kpool) + base);
    const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.vpool) + base);
    const int g = lane / 4, t = lane % 4;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) b.k[n][c] = __ldcs(kp + (8 * n + g) * (D / 8) + c * 4 + t);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) b.v[r][c] = __ldcs(vp + (2 * t + (r & 1) + 8 * (r >> 1)) * (D / 8) + c * 8 + g);
}

template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) few_kernel(AttnArgs a) {
    extern __shared__ __align__(16) float part[];     // [kWarps][kRows][D + 4]
    __shared__ float wm[kWarps][kRows], wl[kWarps][kRows];
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
    const int off = warp * kKeys;

    auto page = [&](int step) -> int32_t {
        const int key = step * kStep + off;
        return key < end ? a.bt[key / a.P] : -1;
    };
    Block<D> x, y;
    int32_t next = page(b0 + 1);
    load_block(x, a, b0 * kStep + off, end, page(b0), kvh, lane);

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

    auto compute = [&](const Block<D>& b) {
        if (b.key0 < 0) return;                       // the same for the whole warp
        float s[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                mma16816(s[nt], q[2 * c], b.k[nt][c].x, b.k[nt][c].y);
                mma16816(s[nt], q[2 * c + 1], b.k[nt][c].z, b.k[nt][c].w);
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
            const int u = (e & 3) >> 1, key = b.key0 + 8 * (e >> 2) + 2 * t + (e & 1);
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
            const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&b.v[0][c]);
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&b.v[1][c]);
            const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&b.v[2][c]);
            const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&b.v[3][c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t sel = j & 1 ? 0x7632 : 0x5410;          // high or low halves of two keys
                mma16816(o[8 * c + j], pw, __byte_perm(w0[j >> 1], w1[j >> 1], sel),
                         __byte_perm(w2[j >> 1], w3[j >> 1], sel));
            }
        }
    };
    for (int b = b0; b < b1; b += 2) {
        load_block(y, a, b + 1 < b1 ? (b + 1) * kStep + off : end, end, next, kvh, lane);
        next = page(b + 2);
        compute(x);
        load_block(x, a, b + 2 < b1 ? (b + 2) * kStep + off : end, end, next, kvh, lane);
        next = page(b + 3);
        compute(y);
    }

    // The warps' states meet: row r's maximum, sum and O.
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
    constexpr int smem = kWarps * kRows * (D + 4) * (int)sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)((a.n_q * (a.Hq / a.Hkv) + kRows - 1) / kRows);
    ProfScope ps("few_kernel", s);
    few_kernel<D><<<dim3(tiles, a.Hkv, a.splits), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Up to 16 queries: their 16-row tiles read each key ceil(n_q g / 16) times (from
// L2 but for the first), the tensor-core kernel's 128-row tiles once per head.
bool few_supported(const AttnArgs& a) {
    return a.dtype == PKV_BF16 && !a.sel && a.n_q <= 16 && a.P % kKeys == 0;
}

int attn_few_splits(const AttnArgs& a) {
    // One wave of CTAs, each with a step of 128 keys at least; up to 4 steps are
    // not worth a second kernel.
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t ctas = (a.n_q * (a.Hq / a.Hkv) + kRows - 1) / kRows * a.Hkv, steps = (a.m.n_keys + kStep - 1) / kStep;
    const int64_t room = std::max<int64_t>(1, sms * (a.d == 64 ? 2 : 1) / ctas);
    return steps <= 4 ? 1 : (int)std::min<int64_t>({steps, room, 512});
}

cudaError_t launch_attn_few(const AttnArgs& a, cudaStream_t s) {
    return a.d == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace pkv
