// Joins the partial results of a forward whose keys were split over CTAs:
//   LSE = log2 sum_s 2^(LSE_s),  O = sum_s 2^(LSE_s - LSE) O_s.
// One warp per (head, query): D / 32 columns per lane, 4 bytes (fp32) each per
// split read once. Splits that saw nothing have LSE_s = -inf and weigh 0.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const float* part, int splits, int Hq, int64_t n_q, T* o,
                                                            float* lse) {
    constexpr int C = D / 32;
    const int lane = threadIdx.x % 32;
    const int64_t rows = (int64_t)Hq * n_q;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;   // h * n_q + i
    if (row >= rows) return;
    const float* l2 = part + (size_t)splits * rows * D + row;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, l2[(size_t)s * rows]);
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float acc[C], sum = 0.f;
#pragma unroll
    for (int e = 0; e < C; ++e) acc[e] = 0.f;
    const float ref = top == -INFINITY ? 0.f : top;
    for (int s = 0; s < splits; ++s) {
        const float w = exp2f(l2[(size_t)s * rows] - ref);
        sum += w;
        if (w == 0.f) continue;
        const float* src = part + ((size_t)s * rows + row) * D + lane * C;
#pragma unroll
        for (int e = 0; e < C; ++e) acc[e] = fmaf(w, src[e], acc[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t h = row / n_q, i = row - h * n_q;
    T* dst = o + ((size_t)i * Hq + h) * D + lane * C;
#pragma unroll
    for (int e = 0; e < C; ++e) Elem<T>::store(dst + e, acc[e] * inv);
    if (lane == 0) lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.Hq * a.n_q;
    ProfScope ps("attn_join_kernel", s);
    attn_join_kernel<T, D><<<(unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s>>>(
        a.part, a.splits, a.Hq, a.n_q, static_cast<T*>(a.o), a.lse);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, cudaStream_t s) {
    if (a.dtype == PKV_BF16) return a.d == 128 ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 64>(a, s);
    return a.d == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
}

}  // namespace pkv
