// Linear attention with a decay per head (lin.cuh) on the CUDA cores: fp32, and
// bf16 where PKV_FLAG_SIMT_ONLY asks for it. All products are float32.
//
// Three launches each way. Forward: each chunk's sum of k v^T, the scan that turns the
// sums into the states before the chunks, and the rows (O). Backward: both kinds of sums,
// both scans, and the rows (dQ) beside the columns (dK, dV). Tiles of 64 rows
// lie in shared memory as float32, rows padded by four words: reads of four words
// along a row are then free of bank conflicts, whether lanes walk rows or columns. A
// thread owns a 4 x (N / 16) patch of a product of 64 x N and reads four inner indices
// (or columns) at a time. Two tiles and the scores are held at most, for two CTAs an SM
// or more. 8 / 2 heads of d 128, 8192 rows in fp32: forward 156 us, backward 410 (268 and
// 676 with single words read and three tiles held); the rows' products run at 37 of the
// fp32 pipes' 80 TFLOP/s. Small calls are bound by the launches' latency: 2 / 1 heads of
// d 64, 201 tokens, both ways 50 us in six launches (82 in nine).
#include <cuda_bf16.h>

#include <type_traits>

#include "lin.cuh"

namespace pkv {
namespace {

constexpr int kL = kLinSimtChunk;
constexpr int kThreads = 256;

constexpr int kLW = 64 + 4;                      // words between rows of 64 columns
template <int D> constexpr int kLD = D + 4;      // and of D
// Words of a tile, which also holds 64 rows of a state, transposed ([D][64]).
template <int D> constexpr int kTile = D * kLW > kL * kLD<D> ? D * kLW : kL * kLD<D>;

__device__ __forceinline__ float4& at4(float* p) { return *reinterpret_cast<float4*>(p); }
__device__ __forceinline__ const float4& at4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// rows x D of one head -> float32 [64][D + 4], zero behind the last row.
template <typename T, int D>
__device__ __forceinline__ void load_tile(float* dst, const LinRows& x, int64_t row0, int rows, int head) {
    constexpr int EPV = 16 / (int)sizeof(T), VPR = D / EPV;
#pragma unroll
    for (int i = threadIdx.x; i < kL * VPR; i += kThreads) {
        const int r = i / VPR, v = i % VPR;
        float f[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) f[e] = 0.f;
        if (r < rows)
            widen16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(x.p) + (row0 + r) * x.stride + (int64_t)head * D) + v), f);
#pragma unroll
        for (int e = 0; e < EPV; e += 4) at4(dst + r * kLD<D> + v * EPV + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
}

// Rows z .. z + 63 of a state: as they are, [64][D + 4], or transposed, [D][64 + 4].
template <int D> __device__ __forceinline__ void load_state(float* dst, const float* S, int z) {
#pragma unroll 8
    for (int i = threadIdx.x; i < 64 * D / 4; i += kThreads) at4(dst + i / (D / 4) * kLD<D> + i % (D / 4) * 4) = at4(S + z * D + 4 * i);
}
template <int D> __device__ __forceinline__ void load_state_t(float* dst, const float* S, int z) {
#pragma unroll 8
    for (int i = threadIdx.x; i < 64 * D / 4; i += kThreads) {
        const int j = i % 64, k = i / 64 * 4;    // (lanes along j: the stores are free of conflicts)
        const float4 x = at4(S + (z + j) * D + k);
        dst[k * kLW + j] = x.x;
        dst[(k + 1) * kLW + j] = x.y;
        dst[(k + 2) * kLW + j] = x.z;
        dst[(k + 3) * kLW + j] = x.w;
    }
}

__device__ __forceinline__ float part_of(const float4& x, int e) { return e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w; }

// x[r][c] += sum_k A[4 ty + r][k] B[tx + 16 c][k]
__device__ __forceinline__ void product_rows(float (&x)[4][4], const float* A, int la, const float* B, int lb, int K) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 p[4], q[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = at4(A + (4 * ty + r) * la + k);
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = at4(B + (tx + 16 * c) * lb + k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[r][c] = fmaf(p[r].x, q[c].x, x[r][c]);
                x[r][c] = fmaf(p[r].y, q[c].y, x[r][c]);
                x[r][c] = fmaf(p[r].z, q[c].z, x[r][c]);
                x[r][c] = fmaf(p[r].w, q[c].w, x[r][c]);
            }
    }
}
// acc[r][4 c + e] += sum_k A[4 ty + r][k] B[k][4 tx + e + 64 c], of columns 4 (C0 ..) to TN - 1 of acc
template <int TN, int C0 = 0, int N>
__device__ __forceinline__ void product(float (&acc)[4][N], const float* A, int la, const float* B, int lb, int K) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = at4(A + (4 * ty + r) * la + k);
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < TN / 4; ++c) {
                const float4 q = at4(B + (k + u) * lb + 4 * tx + 64 * c);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][4 * (C0 + c) + e] = fmaf(part_of(p[r], u), part_of(q, e), acc[r][4 * (C0 + c) + e]);
            }
    }
}
// acc[r][4 c + e] += sum_k w[k] A[k][4 ty + r] B[k][4 tx + e + 64 c], w null: 1
template <int TN>
__device__ __forceinline__ void product_t(float (&acc)[4][TN], const float* A, int la, const float* w, const float* B, int lb, int K) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float4 p = at4(A + k * la + 4 * ty);
        if (w) p = make_float4(p.x * w[k], p.y * w[k], p.z * w[k], p.w * w[k]);
#pragma unroll
        for (int c = 0; c < TN / 4; ++c) {
            const float4 q = at4(B + k * lb + 4 * tx + 64 * c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][4 * c + e] = fmaf(part_of(p, r), part_of(q, e), acc[r][4 * c + e]);
        }
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
    extern __shared__ __align__(16) float sm[];
    constexpr int LD = kLD<D>;
    float *A = sm, *R = sm + kL * LD;
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
        product_t(acc, A + 64 * z, LD, w, R, LD, kL);
    }
    float* out = (grad ? a.gpart : a.part) + ((size_t)blockIdx.x * a.Hkv + h) * D * D;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int cc = 0; cc < D / 16; cc += 4)
            at4(out + (64 * z + 4 * ty + r) * D + 4 * tx + 16 * cc) = make_float4(acc[r][cc], acc[r][cc + 1], acc[r][cc + 2], acc[r][cc + 3]);
}

// Turns a sequence's chunk sums into the states before its chunks (in order) or the
// gradients of the states after them (grad, in reverse), in place. A thread owns four
// elements of a state all along, so slot_in may be slot_out, and has kScanAhead chunks'
// sums on their way at once.
constexpr int kScanAhead = 8;
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
    const int64_t nc = (hi - lo + L - 1) / L;
    const float lfull = lin_pow(g2, L), ltail = lin_pow(g2, (int)(hi - lo - (nc - 1) * L));      // the last chunk's rows
    const int64_t step = (int64_t)a.Hkv * V * (grad ? -1 : 1);
    float4* p = reinterpret_cast<float4*>(grad ? a.gpart : a.part) + ((lo / L + b + (grad ? nc - 1 : 0)) * a.Hkv + h) * V + e;
    for (int64_t i = 0; i < nc; i += kScanAhead, p += kScanAhead * step) {
        float4 x[kScanAhead];
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u)
            if (i + u < nc) x[u] = p[u * step];
#pragma unroll
        for (int u = 0; u < kScanAhead; ++u)
            if (i + u < nc) {
                p[u * step] = s;
                const float l = i + u == (grad ? 0 : nc - 1) ? ltail : lfull;
                s.x = fmaf(l, s.x, x[u].x); s.y = fmaf(l, s.y, x[u].y);
                s.z = fmaf(l, s.z, x[u].z); s.w = fmaf(l, s.w, x[u].w);
            }
    }
    if (last >= 0) reinterpret_cast<float4*>(store + ((size_t)last * a.Hkv + h) * D * D)[e] = s;
}

// The thread's patch of a chunk's rows of one head, times f.
template <typename T, int D>
__device__ __forceinline__ void store_patch(const LinRows& o, const float (&acc)[4][D / 16], float f, const LinChunk& c, int head) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * ty + r < c.rows) {
            T* row = static_cast<T*>(o.p) + (c.row0 + 4 * ty + r) * o.stride + (int64_t)head * D + 4 * tx;
#pragma unroll
            for (int cc = 0; cc < D / 16; cc += 4) {
                const float4 x = make_float4(acc[r][cc] * f, acc[r][cc + 1] * f, acc[r][cc + 2] * f, acc[r][cc + 3] * f);
                if constexpr (sizeof(T) == 4) at4(row + 16 * cc) = x;
                else *reinterpret_cast<uint2*>(row + 16 * cc) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
            }
        }
}

// Rows: out = scale [((X C^T) o M) R + diag(l^(i+1)) X S'], one chunk of one query head.
// O: X = Q, C = K, R = V, S' = S. dQ (GRAD): X = dO, C = V, R = K, S' = S^T.
template <typename T, int D, bool GRAD> __device__ __forceinline__ void rows(const LinArgs& a, int f, int hq) {
    extern __shared__ __align__(16) float sm[];
    constexpr int LD = kLD<D>;
    float *X = sm, *C = X + kL * LD, *W = C + kTile<D>;      // C: C, then S', then R
    __shared__ float pw[kL + 1];
    LinChunk c;
    const int h = hq / (a.Hq / a.Hkv);
    if (!lin_chunk<kL>(a, f, c)) return;
    const float g2 = lin_g2(a, h);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    if (threadIdx.x <= kL) pw[threadIdx.x] = lin_pow(g2, threadIdx.x);
    load_tile<T, D>(X, GRAD ? a.dout : a.q, c.row0, c.rows, hq);
    load_tile<T, D>(C, GRAD ? a.v : a.k, c.row0, c.rows, h);
    __syncthreads();
    {
        float x[4][4];
        clear(x);
        product_rows(x, X, LD, C, LD, D);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                const int i = 4 * ty + r, j = tx + 16 * cc;
                W[i * kLW + j] = j <= i ? x[r][cc] * pw[i - j] : 0.f;
            }
    }
    // X S', the state in pieces of 64 rows: those are the product's inner index, or its columns.
    float acc[4][D / 16];
    clear(acc);
    const float* S = a.part + ((size_t)f * a.Hkv + h) * D * D;
    auto piece = [&](auto z64) {
        constexpr int Z = decltype(z64)::value;
        __syncthreads();
        if (GRAD) load_state_t<D>(C, S, 64 * Z);
        else load_state<D>(C, S, 64 * Z);
        __syncthreads();
        if (GRAD) product<4, Z>(acc, X, LD, C, kLW, D);
        else product<D / 16>(acc, X + 64 * Z, LD, C, LD, 64);
    };
    piece(std::integral_constant<int, 0>());
    if constexpr (D == 128) piece(std::integral_constant<int, 1>());
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int cc = 0; cc < D / 16; ++cc) acc[r][cc] *= pw[4 * ty + r + 1];
    __syncthreads();
    load_tile<T, D>(C, GRAD ? a.k : a.v, c.row0, c.rows, h);
    __syncthreads();
    product<D / 16>(acc, W, kLW, C, LD, kL);
    const float scale = rsqrtf((float)D);
    store_patch<T, D>(GRAD ? a.dq : a.o, acc, scale, c, hq);
}

// Columns: out = scale sum_heads ((X C^T) o M)^T R + diag(l^(m-1-j)) C G', one chunk of one KV head.
// dV: X = Q, C = K, R = dO, G' = G. dK: X = dO, C = V, R = Q, G' = G^T.
template <typename T, int D> __device__ __forceinline__ void cols(const LinArgs& a, int f, int h, bool dk) {
    extern __shared__ __align__(16) float sm[];
    constexpr int LD = kLD<D>;
    float *C = sm, *X = C + kL * LD, *W = X + kTile<D>;      // X: G', then each head's X and R; W: queries x keys
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
    auto piece = [&](auto z64) {
        constexpr int Z = decltype(z64)::value;
        __syncthreads();
        if (dk) load_state_t<D>(X, G, 64 * Z);
        else load_state<D>(X, G, 64 * Z);
        __syncthreads();
        if (dk) product<4, Z>(acc, C, LD, X, kLW, D);
        else product<D / 16>(acc, C + 64 * Z, LD, X, LD, 64);
    };
    piece(std::integral_constant<int, 0>());
    if constexpr (D == 128) piece(std::integral_constant<int, 1>());
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
        __syncthreads();
        float x[4][4];
        clear(x);
        product_rows(x, X, LD, C, LD, D);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                const int i = 4 * ty + r, j = tx + 16 * cc;
                W[i * kLW + j] = j <= i ? x[r][cc] * pw[i - j] * scale : 0.f;
            }
        __syncthreads();
        load_tile<T, D>(X, dk ? a.q : a.dout, c.row0, c.rows, h * g + e);
        __syncthreads();
        product_t(acc, W, kLW, nullptr, X, LD, kL);
    }
    store_patch<T, D>(dk ? a.dk : a.dv, acc, 1.f, c, h);
}

template <typename T, int D> __global__ void __launch_bounds__(kThreads, 2) lin_rows_kernel(LinArgs a) {
    rows<T, D, false>(a, blockIdx.x, blockIdx.y);
}

// The columns first: they are the longer ones.
template <typename T, int D> __global__ void __launch_bounds__(kThreads, 2) lin_grads_kernel(LinArgs a) {
    const int y = blockIdx.x / a.n_chunks, f = blockIdx.x - y * a.n_chunks, c = 2 * a.Hkv;
    if (y < c) cols<T, D>(a, f, y >> 1, y & 1);
    else rows<T, D, true>(a, f, y - c);
}

template <int D> constexpr size_t part_smem() { return 2 * kL * kLD<D> * sizeof(float); }
template <int D> constexpr size_t tile_smem() { return (kL * kLD<D> + kTile<D> + kL * kLW) * sizeof(float); }

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
