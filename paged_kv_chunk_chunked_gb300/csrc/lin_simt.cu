// Linear attention with a decay per head (lin.cuh) on the CUDA cores: fp32, and
// bf16 where PKV_FLAG_SIMT_ONLY asks for it. All products are float32.
//
// Three launches each way. Forward: each chunk's sum of k v^T, the scan that turns the
// sums into the states before the chunks, and the rows (O). Backward: both kinds of sums,
// both scans, and the rows (dQ) beside the columns (dK, dV). Tiles of 64 rows
// lie in shared memory as float32, padded by one word so that walks along either
// dimension are free of bank conflicts; a thread owns a 4 x (N / 16) patch of a
// product of 64 x N. What bounds these kernels is the shared-memory reads of the
// products (12 words for 32 multiply-adds), not HBM.
#include <cuda_bf16.h>

#include "lin.cuh"

namespace pkv {
namespace {

constexpr int kL = kLinSimtChunk;
constexpr int kThreads = 256;

// rows x D of one head -> float32 [64][D + 1], zero behind the last row.
template <typename T, int D>
__device__ __forceinline__ void load_tile(float* dst, const LinRows& x, int64_t row0, int rows, int head) {
    constexpr int EPV = 16 / (int)sizeof(T), VPR = D / EPV;
    for (int i = threadIdx.x; i < kL * VPR; i += kThreads) {
        const int r = i / VPR, v = i % VPR;
        float f[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) f[e] = 0.f;
        if (r < rows)
            widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(x.p) + (row0 + r) * x.stride + (int64_t)head * D) + v), f);
#pragma unroll
        for (int e = 0; e < EPV; ++e) dst[r * (D + 1) + v * EPV + e] = f[e];
    }
}

// acc[r][c] += sum_k A(4 ty + r, k) B(k, tx + 16 c), A and B read by functions.
template <int TN, typename FA, typename FB>
__device__ __forceinline__ void product(float (&acc)[4][TN], int K, FA A, FB B) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float x[4], y[TN];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = A(4 * ty + r, k);
#pragma unroll
        for (int c = 0; c < TN; ++c) y[c] = B(k, tx + 16 * c);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < TN; ++c) acc[r][c] = fmaf(x[r], y[c], acc[r][c]);
    }
}

template <int TN> __device__ __forceinline__ void clear(float (&acc)[4][TN]) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < TN; ++c) acc[r][c] = 0.f;
}

// Chunk sums, rows 64 z .. of the state: sum_j l^(m-1-j) k_j v_j^T, in the second half
// of a backward also scale sum_i l^(i+1) q_i do_i^T over the group's query heads (grad).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) lin_part_kernel(LinArgs a) {
    extern __shared__ float sm[];
    float* A = sm;                               // [64][D + 1]
    float* R = sm + kL * (D + 1);
    __shared__ float w[kL];
    LinChunk c;
    const int h = blockIdx.y, z = blockIdx.z % (D / 64);
    const bool grad = blockIdx.z >= D / 64;
    if (!lin_chunk<kL>(a, blockIdx.x, c)) return;
    const float g2 = lin_g2(a, h);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    if (threadIdx.x < kL)
        w[threadIdx.x] = threadIdx.x >= c.rows ? 0.f
                         : grad ? rsqrtf((float)D) * lin_pow(g2, threadIdx.x + 1) : lin_pow(g2, c.rows - 1 - threadIdx.x);
    float acc[4][D / 16];
    clear(acc);
    const int g = grad ? a.Hq / a.Hkv : 1;
    for (int e = 0; e < g; ++e) {
        __syncthreads();
        load_tile<T, D>(A, grad ? a.q : a.k, c.row0, c.rows, h * g + e);
        load_tile<T, D>(R, grad ? a.dout : a.v, c.row0, c.rows, h * g + e);
        __syncthreads();
        product<D / 16>(acc, kL, [&](int i, int k) { return A[k * (D + 1) + 64 * z + i] * w[k]; },
                        [&](int k, int j) { return R[k * (D + 1) + j]; });
    }
    float* out = (grad ? a.gpart : a.part) + ((size_t)blockIdx.x * a.Hkv + h) * D * D;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int cc = 0; cc < D / 16; ++cc) out[(64 * z + 4 * ty + r) * D + tx + 16 * cc] = acc[r][cc];
}

// Turns a sequence's chunk sums into the states before its chunks (in order) or the
// gradients of the states after them (grad, in reverse), in place. A thread owns four
// elements of a state all along, so slot_in may be slot_out.
template <int D>
__global__ void __launch_bounds__(kThreads) lin_scan_kernel(LinArgs a) {
    constexpr int V = D * D / 4, L = kL;
    const bool grad = blockIdx.y;
    const int64_t unit = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t bh = unit / V;
    if (bh >= a.n_seq * a.Hkv) return;
    const int e = (int)(unit % V), h = (int)(bh % a.Hkv);
    const int64_t b = bh / a.Hkv;
    int64_t lo, hi;
    if (!lin_range(a, b, lo, hi)) return;
    const float g2 = lin_g2(a, h);
    // (a backward scans k v^T for the states alone: the forward has stored the last one)
    const int32_t *from = grad ? a.slot_out : a.slot_in, *to = grad ? a.slot_in : gridDim.y > 1 ? nullptr : a.slot_out;
    const int64_t first = lin_slot(a, from, b), last = lin_slot(a, to, b);
    if (blockIdx.x % (V / kThreads * a.Hkv) == 0) lin_check_alone(a, to, from, b, last, a.n_seq);
    float* store = grad ? a.dstate : a.state;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first >= 0) s = reinterpret_cast<const float4*>(store + ((size_t)first * a.Hkv + h) * D * D)[e];
    const int64_t nc = (hi - lo + L - 1) / L, f0 = lo / L + b;
    float4* part = reinterpret_cast<float4*>(grad ? a.gpart : a.part);
    for (int64_t i = 0; i < nc; ++i) {
        const int64_t c = grad ? nc - 1 - i : i;
        const int m = (int)min64(L, hi - lo - c * L);
        const float l = lin_pow(g2, m);
        float4* p = part + ((size_t)(f0 + c) * a.Hkv + h) * V + e;
        const float4 x = *p;
        *p = s;
        s.x = fmaf(l, s.x, x.x); s.y = fmaf(l, s.y, x.y);
        s.z = fmaf(l, s.z, x.z); s.w = fmaf(l, s.w, x.w);
    }
    if (last >= 0) reinterpret_cast<float4*>(store + ((size_t)last * a.Hkv + h) * D * D)[e] = s;
}

// Rows: out = scale [((X C^T) o M) R + diag(l^(i+1)) X S'], one chunk of one query head.
// O: X = Q, C = K, R = V, S' = S. dQ (GRAD): X = dO, C = V, R = K, S' = S^T.
template <typename T, int D, bool GRAD> __device__ __forceinline__ void rows(const LinArgs& a, int f, int hq) {
    extern __shared__ float sm[];
    constexpr int LD = D + 1;
    float *X = sm, *C = X + kL * LD, *R = C + kL * LD, *W = R + kL * LD;    // W [64][65]
    __shared__ float pw[kL + 1];
    LinChunk c;
    const int h = hq / (a.Hq / a.Hkv);
    if (!lin_chunk<kL>(a, f, c)) return;
    const float g2 = lin_g2(a, h);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    if (threadIdx.x <= kL) pw[threadIdx.x] = lin_pow(g2, threadIdx.x);
    load_tile<T, D>(X, GRAD ? a.dout : a.q, c.row0, c.rows, hq);
    load_tile<T, D>(C, GRAD ? a.v : a.k, c.row0, c.rows, h);
    load_tile<T, D>(R, GRAD ? a.k : a.v, c.row0, c.rows, h);
    __syncthreads();
    {
        float x[4][4];
        clear(x);
        product<4>(x, D, [&](int i, int k) { return X[i * LD + k]; }, [&](int k, int j) { return C[j * LD + k]; });
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                const int i = 4 * ty + r, j = tx + 16 * cc;
                W[i * 65 + j] = j <= i ? x[r][cc] * pw[i - j] : 0.f;
            }
    }
    // X S', the state in pieces of 64 rows over C's place.
    float acc[4][D / 16];
    clear(acc);
    const float* S = a.part + ((size_t)f * a.Hkv + h) * D * D;
    for (int z = 0; z < D; z += 64) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * D; i += kThreads) C[i / D * LD + i % D] = S[z * D + i];
        __syncthreads();
        if (!GRAD) {                             // S rows z .. are the product's inner index
            product<D / 16>(acc, 64, [&](int i, int k) { return X[i * LD + z + k]; },
                            [&](int k, int j) { return C[k * LD + j]; });
        } else {                                 // they are its columns z ..: 4 of a thread's D / 16
            float part[4][4];
            clear(part);
            product<4>(part, D, [&](int i, int k) { return X[i * LD + k]; }, [&](int k, int j) { return C[j * LD + k]; });
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc)
                if (cc / 4 == z / 64)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r][cc] = part[r][cc % 4];
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int cc = 0; cc < D / 16; ++cc) acc[r][cc] *= pw[4 * ty + r + 1];
    product<D / 16>(acc, kL, [&](int i, int k) { return W[i * 65 + k]; }, [&](int k, int j) { return R[k * LD + j]; });
    const float scale = rsqrtf((float)D);
    const LinRows& o = GRAD ? a.dq : a.o;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * ty + r < c.rows) {
            T* row = static_cast<T*>(o.p) + (c.row0 + 4 * ty + r) * o.stride + (int64_t)hq * D;
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc) Elem<T>::store(row + tx + 16 * cc, acc[r][cc] * scale);
        }
}

// Columns: out = scale sum_heads ((X C^T) o M)^T R + diag(l^(m-1-j)) C G', one chunk of one KV head.
// dV: X = Q, C = K, R = dO, G' = G. dK: X = dO, C = V, R = Q, G' = G^T.
template <typename T, int D> __device__ __forceinline__ void cols(const LinArgs& a, int f, int h, bool dk) {
    extern __shared__ float sm[];
    constexpr int LD = D + 1;
    float *C = sm, *X = C + kL * LD, *R = X + kL * LD, *W = R + kL * LD;    // W [64][65]: queries x keys
    __shared__ float pw[kL + 1];
    LinChunk c;
    const int g = a.Hq / a.Hkv;
    if (!lin_chunk<kL>(a, f, c)) return;
    const float g2 = lin_g2(a, h), scale = rsqrtf((float)D);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    if (threadIdx.x <= kL) pw[threadIdx.x] = lin_pow(g2, threadIdx.x);
    load_tile<T, D>(C, dk ? a.v : a.k, c.row0, c.rows, h);
    float acc[4][D / 16];
    clear(acc);
    const float* G = a.gpart + ((size_t)f * a.Hkv + h) * D * D;
    for (int z = 0; z < D; z += 64) {
        __syncthreads();
        for (int i = threadIdx.x; i < 64 * D; i += kThreads) X[i / D * LD + i % D] = G[z * D + i];
        __syncthreads();
        if (!dk) {
            product<D / 16>(acc, 64, [&](int i, int k) { return C[i * LD + z + k]; },
                            [&](int k, int j) { return X[k * LD + j]; });
        } else {
            float part[4][4];
            clear(part);
            product<4>(part, D, [&](int i, int k) { return C[i * LD + k]; }, [&](int k, int j) { return X[j * LD + k]; });
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc)
                if (cc / 4 == z / 64)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r][cc] = part[r][cc % 4];
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = 4 * ty + r;
        const float w = j < c.rows ? pw[c.rows - 1 - j] : 0.f;
#pragma unroll
        for (int cc = 0; cc < D / 16; ++cc) acc[r][cc] *= w;
    }
    for (int e = 0; e < g; ++e) {
        __syncthreads();
        load_tile<T, D>(X, dk ? a.dout : a.q, c.row0, c.rows, h * g + e);
        load_tile<T, D>(R, dk ? a.q : a.dout, c.row0, c.rows, h * g + e);
        __syncthreads();
        float x[4][4];
        clear(x);
        product<4>(x, D, [&](int i, int k) { return X[i * LD + k]; }, [&](int k, int j) { return C[j * LD + k]; });
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                const int i = 4 * ty + r, j = tx + 16 * cc;
                W[i * 65 + j] = j <= i ? x[r][cc] * pw[i - j] * scale : 0.f;
            }
        __syncthreads();
        product<D / 16>(acc, kL, [&](int j, int k) { return W[k * 65 + j]; }, [&](int k, int jj) { return R[k * LD + jj]; });
    }
    const LinRows& o = dk ? a.dk : a.dv;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * ty + r < c.rows) {
            T* row = static_cast<T*>(o.p) + (c.row0 + 4 * ty + r) * o.stride + (int64_t)h * D;
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc) Elem<T>::store(row + tx + 16 * cc, acc[r][cc]);
        }
}

template <typename T, int D> __global__ void __launch_bounds__(kThreads) lin_rows_kernel(LinArgs a) {
    rows<T, D, false>(a, blockIdx.x, blockIdx.y);
}

// The columns first: they are the longer ones.
template <typename T, int D> __global__ void __launch_bounds__(kThreads) lin_grads_kernel(LinArgs a) {
    const int y = blockIdx.x / a.n_chunks, f = blockIdx.x - y * a.n_chunks, c = 2 * a.Hkv;
    if (y < c) cols<T, D>(a, f, y >> 1, y & 1);
    else rows<T, D, true>(a, f, y - c);
}

template <int D> constexpr size_t part_smem() { return 2 * kL * (D + 1) * sizeof(float); }
template <int D> constexpr size_t tile_smem() { return (3 * kL * (D + 1) + kL * 65) * sizeof(float); }

// Each way: the chunks' sums and their scans, of a backward both kinds, then what follows from the states.
template <typename T, int D> cudaError_t run(const LinArgs& a, bool bwd, cudaStream_t s) {
    static SmemGrant part_grant, fwd_grant, bwd_grant;
    const int kinds = bwd ? 2 : 1;
    cudaError_t e = allow_smem(lin_part_kernel<T, D>, part_smem<D>(), part_grant);
    if (e == cudaSuccess)
        e = bwd ? allow_smem(lin_grads_kernel<T, D>, tile_smem<D>(), bwd_grant) : allow_smem(lin_rows_kernel<T, D>, tile_smem<D>(), fwd_grant);
    if (e != cudaSuccess) return e;
    if (a.n) {
        ProfScope ps("lin_part_kernel", s);
        lin_part_kernel<T, D><<<dim3(a.n_chunks, a.Hkv, D / 64 * kinds), kThreads, part_smem<D>(), s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    {
        ProfScope ps("lin_scan_kernel", s);
        lin_scan_kernel<D><<<dim3((unsigned)(a.n_seq * a.Hkv * (D * D / 4 / kThreads)), kinds), kThreads, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess || !a.n) return e;
    }
    ProfScope ps(bwd ? "lin_grads_kernel" : "lin_rows_kernel", s);
    if (bwd) lin_grads_kernel<T, D><<<(unsigned)((int64_t)a.n_chunks * (2 * a.Hkv + a.Hq)), kThreads, tile_smem<D>(), s>>>(a);
    else lin_rows_kernel<T, D><<<dim3(a.n_chunks, a.Hq), kThreads, tile_smem<D>(), s>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t by_d(const LinArgs& a, bool bwd, cudaStream_t s) {
    return a.d == 128 ? run<T, 128>(a, bwd, s) : run<T, 64>(a, bwd, s);
}
cudaError_t by_type(const LinArgs& a, bool bwd, cudaStream_t s) {
    return a.dtype == PKV_BF16 ? by_d<__nv_bfloat16>(a, bwd, s) : by_d<float>(a, bwd, s);
}

}  // namespace

cudaError_t launch_lin_fwd_simt(const LinArgs& a, cudaStream_t s) { return by_type(a, false, s); }
cudaError_t launch_lin_bwd_simt(const LinArgs& a, cudaStream_t s) { return by_type(a, true, s); }

}  // namespace pkv
