// Layer norm over groups of columns, forward and backward.
//
//   y = xhat w + b, xhat = (x - mean) rstd;   with u = w dy:
//   dx = rstd (u - mean(u) - xhat mean(u xhat)),   dw = sum_rows dy xhat,   db = sum_rows dy.
// The variance is the mean square of x - mean, from the values in registers: no
// cancellation for rows whose mean is far from zero.
//
// One pass over HBM each way: a team of threads holds a group's columns in
// registers, kEPV at a time (16-byte vectors, or single elements where rows are
// not whole vectors). A team is 1 to 32 lanes (sums by shuffles) or, for more
// than 1024 columns, a CTA. In the backward a team keeps to one group of columns
// and walks rows, so its share of dw and db stays in registers; the shares
// are added by a second kernel in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;                    // of a CTA of lane teams
constexpr int64_t kMaxWidth = 32768, kMaxGrid = (int64_t(1) << 31) - 1;

struct NormArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx;                                // y: forward
    int64_t xs, dys, ys, dxs;                    // elements between rows
    float *mean, *rstd, *dw, *db, *part;         // part: [slots][2][groups * width]
    int64_t n;
    int groups, width;
    int team;                                    // lanes of a team, or kThreads' whole CTA: blockDim.x
    int slots;                                   // backward: teams that share a group's rows
    float eps;
    bool w_f32, accumulate;
};

template <typename T, int EPV> __device__ __forceinline__ void load(const T* p, float* f) {
    if constexpr (EPV == 1) {
        f[0] = Elem<T>::load(p);
    } else {
        widen16<T>(*reinterpret_cast<const uint4*>(p), f);
    }
}
template <typename T, int EPV> __device__ __forceinline__ void store(T* p, const float* f) {
    if constexpr (EPV == 1) {
        Elem<T>::store(p, f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                                  pack_bf16x2(f[6], f[7]));
    }
}
// Weight or bias, EPV columns from c on; `none` where there is none.
template <int EPV> __device__ __forceinline__ void load_w(const void* w, bool f32, int64_t c, float none, float* f) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) f[e] = none;
    } else if (f32) {
        const float* p = static_cast<const float*>(w) + c;
        if constexpr (EPV == 1) {
            f[0] = *p;
        } else {
#pragma unroll
            for (int e = 0; e < EPV; e += 4) widen16<float>(*reinterpret_cast<const uint4*>(p + e), f + e);
        }
    } else {
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w) + c;
        if constexpr (EPV == 1) {
            f[0] = __bfloat162float(*p);
        } else if constexpr (EPV == 8) {
            widen16<__nv_bfloat16>(*reinterpret_cast<const uint4*>(p), f);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
        }
    }
}

// Sum of x over the team (CTA: the whole CTA, which all its threads call).
template <bool CTA> __device__ __forceinline__ float2 team_sum(float2 x, int team, float2* red) {
    const int lanes = CTA ? 32 : team;
    for (int d = 1; d < lanes; d *= 2) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, d);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, d);
    }
    if (CTA) {
        __syncthreads();                         // the last sum has been read
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
        __syncthreads();
        x = make_float2(0.f, 0.f);
        for (int i = 0; i < (int)blockDim.x / 32; ++i) {
            x.x += red[i].x;
            x.y += red[i].y;
        }
    }
    return x;
}

template <typename T, int EPV, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : kThreads) layer_norm_fwd_kernel(NormArgs a) {
    __shared__ float2 red[32];
    const int team = CTA ? (int)blockDim.x : a.team, t = CTA ? (int)threadIdx.x : (int)threadIdx.x % team;
    const int64_t unit = CTA ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x * kThreads + threadIdx.x) / team;
    const bool live = unit < a.n * a.groups;
    const int64_t row = unit / a.groups;
    const int64_t c0 = (unit % a.groups) * a.width;
    const T* x = static_cast<const T*>(a.x) + row * a.xs + c0;
    float f[NV][EPV];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (t + v * team) * EPV;
        const bool in = live && c < a.width;
        if (in) load<T, EPV>(x + c, f[v]);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            if (!in) f[v][e] = 0.f;
            s.x += f[v][e];
        }
    }
    const float mean = team_sum<CTA>(s, team, red).x / (float)a.width;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            f[v][e] -= mean;
            if ((t + v * team) * EPV < a.width) s.x = fmaf(f[v][e], f[v][e], s.x);
        }
    const float rstd = 1.f / sqrtf(team_sum<CTA>(s, team, red).x / (float)a.width + a.eps);
    if (!live) return;
    if (t == 0 && a.mean) {
        a.mean[unit] = mean;
        a.rstd[unit] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ys + c0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (t + v * team) * EPV;
        if (c < a.width) {
            float w[EPV], b[EPV];
            load_w<EPV>(a.w, a.w_f32, c0 + c, 1.f, w);
            load_w<EPV>(a.b, a.w_f32, c0 + c, 0.f, b);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[v][e] = fmaf(f[v][e] * rstd, w[e], b[e]);
            store<T, EPV>(y + c, f[v]);
        }
    }
}

// Teams numbered so that neighbours take neighbouring groups of one row.
template <typename T, int EPV, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : kThreads) layer_norm_bwd_kernel(NormArgs a) {
    __shared__ float2 red[32];
    const int team = CTA ? (int)blockDim.x : a.team, t = CTA ? (int)threadIdx.x : (int)threadIdx.x % team;
    const int64_t id = CTA ? (int64_t)blockIdx.x : ((int64_t)blockIdx.x * kThreads + threadIdx.x) / team;
    const int grp = (int)(id % a.groups);
    const int64_t slot = id / a.groups;
    const int64_t c0 = (int64_t)grp * a.width;
    float w[NV][EPV], dw[NV][EPV], db[NV][EPV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (t + v * team) * EPV;
        if (c < a.width) load_w<EPV>(a.w, a.w_f32, c0 + c, 1.f, w[v]);
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            if (c >= a.width) w[v][e] = 0.f;
            dw[v][e] = db[v][e] = 0.f;
        }
    }
    // Every team of a warp makes the same number of rounds: its lanes meet in the sums.
    const int64_t rounds = (a.n + a.slots - 1) / a.slots;
    for (int64_t it = 0; it < rounds; ++it) {
        const int64_t row = it * a.slots + slot;
        const bool live = slot < a.slots && row < a.n;
        const T* x = static_cast<const T*>(a.x) + row * a.xs + c0;
        const T* dy = static_cast<const T*>(a.dy) + row * a.dys + c0;
        float f[NV][EPV], u[NV][EPV];
        float2 s = make_float2(0.f, 0.f);
        const float mean = live ? a.mean[row * a.groups + grp] : 0.f, rstd = live ? a.rstd[row * a.groups + grp] : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (t + v * team) * EPV;
            const bool in = live && c < a.width;
            if (in) {
                load<T, EPV>(x + c, f[v]);
                load<T, EPV>(dy + c, u[v]);
            }
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                f[v][e] = in ? (f[v][e] - mean) * rstd : 0.f;
                if (!in) u[v][e] = 0.f;
                dw[v][e] = fmaf(u[v][e], f[v][e], dw[v][e]);
                db[v][e] += u[v][e];
                u[v][e] *= w[v][e];
                s.x += u[v][e];
                s.y = fmaf(u[v][e], f[v][e], s.y);
            }
        }
        if (!a.dx) continue;
        s = team_sum<CTA>(s, team, red);
        const float m1 = s.x / (float)a.width, m2 = s.y / (float)a.width;
        if (!live) continue;
        T* dx = static_cast<T*>(a.dx) + row * a.dxs + c0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (t + v * team) * EPV;
            if (c < a.width) {
#pragma unroll
                for (int e = 0; e < EPV; ++e) u[v][e] = (u[v][e] - m1 - f[v][e] * m2) * rstd;
                store<T, EPV>(dx + c, u[v]);
            }
        }
    }
    if (!a.part || slot >= a.slots) return;
    const int64_t cols = (int64_t)a.groups * a.width;
    float* pw = a.part + slot * 2 * cols + c0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (t + v * team) * EPV;
        if (c < a.width)
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                pw[c + e] = dw[v][e];
                pw[cols + c + e] = db[v][e];
            }
    }
}

// dw and db from the slots' shares: 32 columns a CTA, 8 runs of slots, added in order.
__global__ void __launch_bounds__(256) layer_norm_sum_kernel(NormArgs a) {
    __shared__ float red[8][33];
    const int64_t cols = (int64_t)a.groups * a.width;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t c = (int64_t)blockIdx.x * 32 + tx;
    float* out = blockIdx.y ? a.db : a.dw;
    if (!out) return;
    float s = 0.f;
    if (c < cols) {
        const float* p = a.part + blockIdx.y * cols + c;
#pragma unroll 8
        for (int r = ty; r < a.slots; r += 8) s += p[(int64_t)r * 2 * cols];
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][tx];
        out[c] = a.accumulate ? out[c] + s : s;
    }
}

// Vectors of a thread and lanes of a team for nvec vectors; a team of more than 32 lanes is a CTA.
struct Shape {
    int nv, team;
};
Shape shape_of(int64_t nvec, int max_nv) {
    int nv = 1;
    if (nvec <= 32) {
        int t = 1;
        while (t < nvec) t *= 2;
        return {1, t};
    }
    while (nv < max_nv && nvec > 32 * nv) nv *= 2;
    if (nvec <= 32 * nv) return {nv, 32};
    nv = 1;
    while (nv < max_nv && nvec > 256 * nv) nv *= 2;
    return {nv, (int)((nvec + 32 * nv - 1) / (32 * nv) * 32)};
}

// Rows shared by a group's teams in the backward: enough teams for two CTAs an SM.
int slots_of(int64_t n, int groups, int team) {
    const int64_t teams = team > 32 ? 304 : 304 * (kThreads / team);
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, (teams + groups - 1) / groups));
}

template <typename T, int EPV, int NV> cudaError_t run(NormArgs& a, bool bwd, int team, cudaStream_t s) {
    const bool cta = team > 32;
    const int64_t units = bwd ? (int64_t)a.slots * a.groups : a.n * a.groups;
    const int64_t grid = cta ? units : (units + kThreads / team - 1) / (kThreads / team);
    if (grid > kMaxGrid) return cudaErrorInvalidConfiguration;
    ProfScope ps(bwd ? "layer_norm_bwd_kernel" : "layer_norm_fwd_kernel", s);
    if (bwd && cta) layer_norm_bwd_kernel<T, EPV, NV, true><<<(unsigned)grid, team, 0, s>>>(a);
    else if (bwd) layer_norm_bwd_kernel<T, EPV, NV, false><<<(unsigned)grid, kThreads, 0, s>>>(a);
    else if (cta) layer_norm_fwd_kernel<T, EPV, NV, true><<<(unsigned)grid, team, 0, s>>>(a);
    else layer_norm_fwd_kernel<T, EPV, NV, false><<<(unsigned)grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t dispatch(NormArgs& a, bool bwd, bool vec, cudaStream_t s) {
    constexpr int EPV = 16 / (int)sizeof(T), MAXV = 32 / EPV;
    const Shape sh = vec ? shape_of(a.width / EPV, MAXV) : shape_of(a.width, 32);
    a.team = sh.team;
    if (vec) {
        if (sh.nv == 1) return run<T, EPV, 1>(a, bwd, sh.team, s);
        if (sh.nv == 2) return run<T, EPV, 2>(a, bwd, sh.team, s);
        if (sh.nv == 4) return run<T, EPV, 4>(a, bwd, sh.team, s);
        if constexpr (MAXV == 8) return run<T, EPV, 8>(a, bwd, sh.team, s);
    }
    return sh.nv <= 8 ? run<T, 1, 8>(a, bwd, sh.team, s) : run<T, 1, 32>(a, bwd, sh.team, s);
}

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

pkv_status norm_args(const pkv_norm* norm, int64_t n, NormArgs* a, const char* who) {
    const std::string w(who);
    if (!norm) return fail(PKV_ERR_INVALID, w + ": norm is NULL");
    if ((norm->dtype != PKV_BF16 && norm->dtype != PKV_F32) || (norm->w_dtype != PKV_BF16 && norm->w_dtype != PKV_F32))
        return fail(PKV_ERR_INVALID, w + ": dtype and w_dtype must be PKV_BF16 or PKV_F32");
    if (norm->groups <= 0 || norm->width <= 0 || !(norm->eps >= 0.f) || norm->eps > 3.4e38f)
        return fail(PKV_ERR_INVALID, w + ": groups and width must be positive, eps a finite number >= 0");
    if (norm->width > kMaxWidth) return fail(PKV_ERR_UNSUPPORTED, w + ": width must be at most 32768");
    if (n < 0 || n > (int64_t(1) << 40) || (n > 0 && norm->groups > (int64_t(1) << 40) / n))
        return fail(PKV_ERR_INVALID, w + ": n out of range");
    const uintptr_t we = norm->w_dtype == PKV_BF16 ? 2 : 4;
    if (misaligned(norm->weight, we) || misaligned(norm->bias, we))
        return fail(PKV_ERR_INVALID, w + ": weight or bias is misaligned");
    a->w = norm->weight; a->b = norm->bias;
    a->w_f32 = norm->w_dtype == PKV_F32;
    a->n = n; a->groups = norm->groups; a->width = (int)norm->width; a->eps = norm->eps;
    return PKV_OK;
}

pkv_status rows(const pkv_norm* norm, const void* x, int64_t* stride, bool* vec, const char* who, const char* name) {
    const int64_t cols = norm->groups * norm->width, e = norm->dtype == PKV_BF16 ? 2 : 4;
    if (*stride == 0) *stride = cols;
    if (!x) return fail(PKV_ERR_INVALID, std::string(who) + ": " + name + " is NULL");
    if (*stride < cols || misaligned(x, e))
        return fail(PKV_ERR_INVALID, std::string(who) + ": " + name + " must be aligned to its type, with rows at least groups * "
                                         "width elements apart");
    if (misaligned(x, 16) || (*stride * e) % 16) *vec = false;
    return PKV_OK;
}

// Whether rows are whole 16-byte vectors, as far as the widths and the weights say.
bool whole_vectors(const pkv_norm* norm) {
    return norm->width % (norm->dtype == PKV_BF16 ? 8 : 4) == 0 && !misaligned(norm->weight, 16) && !misaligned(norm->bias, 16);
}

// The backward's slots do not depend on the addresses: scratch for vectors and for single elements.
int slots_for(const pkv_norm* norm, int64_t n, bool vec) {
    const int epv = norm->dtype == PKV_BF16 ? 8 : 4;
    return slots_of(n, norm->groups, vec ? shape_of(norm->width / epv, 32 / epv).team : shape_of(norm->width, 32).team);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_layer_norm_fwd(const void* x, int64_t x_stride, void* y, int64_t y_stride, float* mean, float* rstd, int64_t n,
                              const pkv_norm* norm, void* stream) {
    static const char* who = "pkv_layer_norm_fwd";
    return guarded(who, [&]() -> pkv_status {
        NormArgs a{};
        pkv_status st = norm_args(norm, n, &a, who);
        if (st != PKV_OK || n == 0) return st;
        bool vec = whole_vectors(norm);
        if ((st = rows(norm, x, &x_stride, &vec, who, "x")) != PKV_OK) return st;
        if ((st = rows(norm, y, &y_stride, &vec, who, "y")) != PKV_OK) return st;
        if (!mean != !rstd || misaligned(mean, 4) || misaligned(rstd, 4))
            return fail(PKV_ERR_INVALID, "pkv_layer_norm_fwd: mean and rstd go together, aligned to float32");
        a.x = x; a.xs = x_stride; a.y = y; a.ys = y_stride; a.mean = mean; a.rstd = rstd;
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        const cudaError_t e = norm->dtype == PKV_BF16 ? dispatch<__nv_bfloat16>(a, false, vec, cs) : dispatch<float>(a, false, vec, cs);
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_layer_norm_fwd: launch");
    });
}

pkv_status pkv_layer_norm_scratch(const pkv_norm* norm, int64_t n, int64_t* floats) {
    static const char* who = "pkv_layer_norm_scratch";
    return guarded(who, [&]() -> pkv_status {
        NormArgs a{};
        const pkv_status st = norm_args(norm, n, &a, who);
        if (st != PKV_OK) return st;
        if (!floats) return fail(PKV_ERR_INVALID, "pkv_layer_norm_scratch: floats is NULL");
        const int64_t cols = norm->groups * norm->width;
        *floats = n == 0 ? 0 : 2 * cols * std::max(slots_for(norm, n, true), slots_for(norm, n, false));
        return PKV_OK;
    });
}

pkv_status pkv_layer_norm_bwd(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, const float* mean,
                              const float* rstd, void* dx, int64_t dx_stride, float* dw, float* db, int32_t accumulate,
                              float* scratch, int64_t n, const pkv_norm* norm, void* stream) {
    static const char* who = "pkv_layer_norm_bwd";
    return guarded(who, [&]() -> pkv_status {
        NormArgs a{};
        pkv_status st = norm_args(norm, n, &a, who);
        if (st != PKV_OK) return st;
        if (accumulate != 0 && accumulate != 1) return fail(PKV_ERR_INVALID, "pkv_layer_norm_bwd: accumulate must be 0 or 1");
        if (misaligned(dw, 4) || misaligned(db, 4)) return fail(PKV_ERR_INVALID, "pkv_layer_norm_bwd: dw or db is misaligned");
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        a.dw = dw; a.db = db; a.accumulate = accumulate != 0;
        bool vec = whole_vectors(norm);
        if (n > 0) {
            if ((st = rows(norm, dy, &dy_stride, &vec, who, "dy")) != PKV_OK) return st;
            if ((st = rows(norm, x, &x_stride, &vec, who, "x")) != PKV_OK) return st;
            if (dx && (st = rows(norm, dx, &dx_stride, &vec, who, "dx")) != PKV_OK) return st;
            if (!mean || !rstd || misaligned(mean, 4) || misaligned(rstd, 4))
                return fail(PKV_ERR_INVALID, "pkv_layer_norm_bwd: mean or rstd is NULL or misaligned");
            if ((dw || db) && (!scratch || misaligned(scratch, 16)))
                return fail(PKV_ERR_INVALID, "pkv_layer_norm_bwd: scratch is NULL or not 16-byte aligned");
            a.dy = dy; a.dys = dy_stride; a.x = x; a.xs = x_stride; a.dx = dx; a.dxs = dx_stride;
            a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
            a.part = dw || db ? scratch : nullptr;
            a.slots = slots_for(norm, n, vec);
            if (!dx && !a.part) return PKV_OK;
            const cudaError_t e = norm->dtype == PKV_BF16 ? dispatch<__nv_bfloat16>(a, true, vec, cs) : dispatch<float>(a, true, vec, cs);
            if (e != cudaSuccess) return cuda_fail(e, "pkv_layer_norm_bwd: launch");
        }
        if (!dw && !db) return PKV_OK;
        // (no rows: dw and db are sums of nothing)
        ProfScope ps("layer_norm_sum_kernel", cs);
        const int64_t cols = norm->groups * norm->width;
        layer_norm_sum_kernel<<<dim3((unsigned)((cols + 31) / 32), 2), 256, 0, cs>>>(a);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_layer_norm_bwd: launch");
    });
}

}  // extern "C"
