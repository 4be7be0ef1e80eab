// Joins the partial results of a forward whose keys were split over CTAs:
//   LSE = log2 sum_s 2^(LSE_s),  O = sum_s 2^(LSE_s - LSE) O_s.
// One CTA per (head, query): the splits' weights once in shared memory, then
// warp w adds splits w, w + 4, ... in a fixed order, 4 bytes (fp32) per element
// and split. Splits that saw nothing have LSE_s = -inf and weigh 0. Latency
// bound (28 rows of 38 splits: 0.5 MB): the grid is launched as a programmatic
// dependent, so that its CTAs stand ready when the forward's last one ends.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kMaxSplits = 512;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const float* part, int splits, int Hq, int64_t n_q, T* o,
                                                            float* lse) {
    constexpr int C = D / 32;
    __shared__ float weight[kMaxSplits], acc_s[kWarps][D], top_s[kWarps], sum_s[kWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t rows = (int64_t)Hq * n_q, row = blockIdx.x;                  // h * n_q + i
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float* l2 = part + (size_t)splits * rows * D + row;
    float top = -INFINITY;
    for (int s = threadIdx.x; s < splits; s += kThreads) {
        weight[s] = l2[(size_t)s * rows];
        top = fmaxf(top, weight[s]);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) top_s[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(top_s[0], top_s[1]), fmaxf(top_s[2], top_s[3]));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int s = threadIdx.x; s < splits; s += kThreads) {
        weight[s] = exp2f(weight[s] - ref);
        sum += weight[s];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) sum_s[warp] = sum;
    __syncthreads();
    sum = (sum_s[0] + sum_s[1]) + (sum_s[2] + sum_s[3]);
    float acc[C];
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int s = warp; s < splits; s += kWarps) {
        const float w = weight[s];
        const float* src = part + ((size_t)s * rows + row) * D + lane * C;
        float x[C];
        if constexpr (C == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[0] = v.x; x[1] = v.y;
        }
#pragma unroll
        for (int e = 0; e < C; ++e) acc[e] = fmaf(w, x[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < C; ++e) acc_s[warp][lane * C + e] = acc[e];
    __syncthreads();
    const int64_t h = row / n_q, i = row - h * n_q;
    const int c = threadIdx.x;
    if (c < D) {
        const float x = (acc_s[0][c] + acc_s[1][c]) + (acc_s[2][c] + acc_s[3][c]);
        Elem<T>::store(o + ((size_t)i * Hq + h) * D + c, sum == 0.f ? 0.f : x / sum);
    }
    if (threadIdx.x == 0) lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    if (a.splits > kMaxSplits) return cudaErrorInvalidValue;
    cudaLaunchAttribute dependent{};
    dependent.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dependent.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)a.Hq * a.n_q));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = &dependent;
    cfg.numAttrs = 1;
    ProfScope ps("attn_join_kernel", s);
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<T, D>, (const float*)a.part, a.splits, a.Hq, a.n_q,
                              static_cast<T*>(a.o), a.lse);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t s) {
    if (a.dtype == PKV_BF16) return a.d == 128 ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 64>(a, s);
    return a.d == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
}

}  // namespace pkv
