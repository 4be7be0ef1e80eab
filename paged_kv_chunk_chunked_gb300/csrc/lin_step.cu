// One token of linear attention for each of n sequences: S <- l S + k v^T in
// place, o = scale q^T S for the group's query heads.
//
// A stream over the states: each is read and written once (8 d^2 bytes per KV
// head for 4 d^2 multiply-adds per query head), so HBM bounds it. A CTA takes 64
// columns of one state, a thread four columns of D / 16 rows, held in registers
// from the load to the last query head's product. Loads and stores are marked as
// streaming (4 us of 25). 187 states of 4 heads of d 128 take 20.1 us (4.9 TB/s) so,
// with 32 columns a CTA 21.5, with 128 21.8; with four query heads at once 20.4. One
// CTA of a row looks for its slot in the rows before (0.7 us).
#include <cuda_bf16.h>

#include "lin.cuh"

namespace pkv {
namespace {

constexpr int kCols = 64, kRowGroups = 16, kLanes = kCols / 4, kThreads = kLanes * kRowGroups, kWarps = kThreads / 32;
constexpr int kHeads = 8;                        // query heads whose partial sums shared memory holds at once

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) lin_step_kernel(LinArgs a) {
    constexpr int R = D / kRowGroups;            // rows of a thread
    static_assert(kLanes <= 32 && D % kCols == 0 && D <= kThreads, "a warp has whole rows of the columns; a thread loads one k");
    __shared__ float ks[D];
    __shared__ float qs[kHeads][D];
    __shared__ float red[kWarps][kHeads][kCols];
    const int64_t i = blockIdx.x / (a.Hkv * (D / kCols));
    const int h = blockIdx.x / (D / kCols) % a.Hkv, c0 = blockIdx.x % (D / kCols) * kCols;
    const int64_t slot = lin_slot(a, a.slots, i);
    if (slot < 0) return;
    const int tid = threadIdx.x, tx = tid % kLanes, rg = tid / kLanes;
    float4* S = reinterpret_cast<float4*>(a.state + ((size_t)slot * a.Hkv + h) * D * D + (size_t)rg * R * D + c0) + tx;
    float4 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = __ldcs(S + r * (D / 4));
    const T* krow = static_cast<const T*>(a.k.p) + i * a.k.stride + (int64_t)h * D;
    const T* vrow = static_cast<const T*>(a.v.p) + i * a.v.stride + (int64_t)h * D + c0 + 4 * tx;
    if (tid < D) ks[tid] = Elem<T>::load(krow + tid);
    const float v0 = Elem<T>::load(vrow), v1 = Elem<T>::load(vrow + 1), v2 = Elem<T>::load(vrow + 2), v3 = Elem<T>::load(vrow + 3);
    const float l = lin_pow(lin_g2(a, h), 1), scale = rsqrtf((float)D);
    const int g = a.Hq / a.Hkv;
    for (int e0 = 0; e0 < g; e0 += kHeads) {
        const int ne = min(kHeads, g - e0);
        const T* qrow = static_cast<const T*>(a.q.p) + i * a.q.stride + (int64_t)(h * g + e0) * D;
        for (int x = tid; x < ne * D; x += kThreads) qs[x / D][x % D] = Elem<T>::load(qrow + x) * scale;
        __syncthreads();
        if (e0 == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float kk = ks[rg * R + r];
                s[r].x = fmaf(l, s[r].x, kk * v0); s[r].y = fmaf(l, s[r].y, kk * v1);
                s[r].z = fmaf(l, s[r].z, kk * v2); s[r].w = fmaf(l, s[r].w, kk * v3);
                __stcs(S + r * (D / 4), s[r]);
            }
        for (int e = 0; e < ne; ++e) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float q = qs[e][rg * R + r];
                o.x = fmaf(q, s[r].x, o.x); o.y = fmaf(q, s[r].y, o.y);
                o.z = fmaf(q, s[r].z, o.z); o.w = fmaf(q, s[r].w, o.w);
            }
#pragma unroll
            for (int d = kLanes; d < 32; d *= 2) {       // the warp's row groups
                o.x += __shfl_xor_sync(0xffffffffu, o.x, d); o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, d); o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
            }
            if (tid % 32 < kLanes) *reinterpret_cast<float4*>(&red[tid / 32][e][4 * tx]) = o;
        }
        __syncthreads();
        T* orow = static_cast<T*>(a.o.p) + i * a.o.stride + (int64_t)(h * g + e0) * D + c0;
        for (int x = tid; x < ne * kCols; x += kThreads) {
            const int e = x / kCols, c = x % kCols;
            float o = red[0][e][c];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) o += red[w][e][c];
            Elem<T>::store(orow + e * D + c, o);
        }
    }
    if (h == 0 && c0 == 0) lin_check_alone(a, a.slots, nullptr, i, slot, a.n);
}

template <typename T, int D> cudaError_t step(const LinArgs& a, cudaStream_t s) {
    ProfScope ps("lin_step_kernel", s);
    lin_step_kernel<T, D><<<(unsigned)(a.n * a.Hkv * (D / kCols)), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lin_step(const LinArgs& a, cudaStream_t s) {
    if (a.dtype == PKV_BF16) return a.d == 128 ? step<__nv_bfloat16, 128>(a, s) : step<__nv_bfloat16, 64>(a, s);
    return a.d == 128 ? step<float, 128>(a, s) : step<float, 64>(a, s);
}

}  // namespace pkv
