// Layer norm over groups of columns, forward and backward.
//
//   y = xhat w + b, xhat = (x - mean) rstd;   with u = w dy:
//   dx = rstd (u - mean(u) - xhat mean(u xhat)),   dw = sum_rows dy xhat,   db = sum_rows dy.
// The variance is the mean square of x - mean, from the values in registers: no
// cancellation for rows whose mean is far from zero.
//
// One pass over HBM each way: a team of threads holds a group's columns in
// registers, as loaded: 16-byte vectors, or single elements where rows are not
// whole vectors. A team is 1 to 32 lanes with a vector each (sums by shuffles) or
// whole warps with several vectors a thread: the sums between warps cost every
// thread two barriers and a read per warp, so few warps a row and many rows at once
// are better than many warps. In the backward a team keeps to one group of columns,
// so that its share of dw and db stays in registers, and walks rows; a CTA's teams
// add their shares in shared memory, a second kernel adds the CTAs', both in a fixed
// order. Rows of more columns than that holds have a backward of two kernels that read x
// and dy twice.
// Replayed on the same buffers (partly in L2), bf16: 4096 rows of 3584 columns forward
// 11.8 us (5.0 TB/s), backward 24.3 (3.6 TB/s; 4.7 of it the second kernel); 28 groups of
// 128 columns 12.0 and 23.2; 2048 rows of 16384 columns 45 and 93. Where rows come from HBM
// the first pair takes 16.6 and 25 us. The sums' latency and issue slots (56% used)
// bound them as much as HBM; a forward CTA that takes several rows and loads the next one
// ahead was slower (13.2 us at best).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mod.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;                    // of a CTA of lane teams
constexpr int kMaxTeam = 512;                    // threads of a CTA of teams of warps, but for the widest rows
// Rows that a team of the backward has on the way: 128 KB of x and dy at most, and none of single
// elements.
template <int EPV, int NV> constexpr int kAhead = EPV == 1 ? 0 : 8 / NV;
constexpr int kBatch = 4;
constexpr int64_t kMaxWidth = 32768, kMaxGrid = (int64_t(1) << 31) - 1;

struct NormArgs {
    const void *x, *dy, *w, *b;
    void *y, *dx;
    int64_t xs, dys, ys, dxs;                    // elements between rows
    float *mean, *rstd, *dw, *db, *part;         // part: [slots][2][groups * width]
    int64_t n;
    int groups, width;
    int team;                                    // threads of a team
    int slots;                                   // lane teams, or CTAs, that share a group's rows
    float eps, inv_width;
    bool w_f32, accumulate;
};

// Elements are worked on in pairs where a vector holds some (f32x2: one instruction
// for two), single ones by the same code.
template <int EPV> using Pk = std::conditional_t<EPV == 1, float, f32x2>;
template <int EPV> constexpr int kPk = EPV == 1 ? 1 : EPV / 2;
using pkv::fma2;                                 // (not hidden by the single ones)
using pkv::mul2;
using pkv::add2;
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
template <typename P> __device__ __forceinline__ P both(float x) {
    if constexpr (std::is_same_v<P, float>) return x;
    else return pack2(x, x);
}
__device__ __forceinline__ float total(float x) { return x; }
__device__ __forceinline__ float total(f32x2 x) {
    float a, b;
    unpack2(x, a, b);
    return a + b;
}
template <int EPV> __device__ __forceinline__ void pairs(const float (&f)[EPV], Pk<EPV> (&p)[kPk<EPV>]) {
    if constexpr (EPV == 1) {
        p[0] = f[0];
    } else {
#pragma unroll
        for (int e = 0; e < EPV / 2; ++e) p[e] = pack2(f[2 * e], f[2 * e + 1]);
    }
}
template <int EPV> __device__ __forceinline__ void singles(const Pk<EPV> (&p)[kPk<EPV>], float (&f)[EPV]) {
    if constexpr (EPV == 1) {
        f[0] = p[0];
    } else {
#pragma unroll
        for (int e = 0; e < EPV / 2; ++e) unpack2(p[e], f[2 * e], f[2 * e + 1]);
    }
}

// EPV consecutive elements as they are in memory.
template <typename T, int EPV> struct Raw {
    uint4 u;
    __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void widen(f32x2 (&p)[EPV / 2]) const {
        float f[EPV];
        widen16<T>(u, f);
        pairs<EPV>(f, p);
    }
};
// 16 bytes global -> shared memory, asynchronously; groups of copies are waited for in order.
__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

template <typename T> struct Raw<T, 1> {
    float x;
    __device__ __forceinline__ void load(const T* p) { x = Elem<T>::load(p); }
    __device__ __forceinline__ void zero() { x = 0.f; }
    __device__ __forceinline__ void widen(float (&p)[1]) const { p[0] = x; }
};
template <typename T, int EPV> __device__ __forceinline__ void store(T* p, const Pk<EPV> (&x)[kPk<EPV>]) {
    float f[EPV];
    singles<EPV>(x, f);
    if constexpr (EPV == 1) {
        Elem<T>::store(p, f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                                  pack_bf16x2(f[6], f[7]));
    }
}
// Weight or bias of type W, EPV columns from c on; `none` where there is none. Read-only
// loads: they may move ahead of the stores of outputs, which could otherwise be the
// weights. (The type is no branch here: in one, each vector's load waited for the one
// before, 9 us for a row of 3584 columns instead of 3.)
template <typename W, int EPV> __device__ __forceinline__ void load_w(const void* w, int64_t c, float none, Pk<EPV> (&x)[kPk<EPV>]) {
#pragma unroll
    for (int e = 0; e < kPk<EPV>; ++e) x[e] = both<Pk<EPV>>(none);
    if (!w) return;
    float f[EPV];
    const W* p = static_cast<const W*>(w) + c;
    if constexpr (EPV == 1) {
        f[0] = (float)__ldg(p);
    } else if constexpr (sizeof(W) == 4) {
#pragma unroll
        for (int e = 0; e < EPV; e += 4) widen16<float>(__ldg(reinterpret_cast<const uint4*>(p + e)), f + e);
    } else if constexpr (EPV == 8) {
        widen16<__nv_bfloat16>(__ldg(reinterpret_cast<const uint4*>(p)), f);
    } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
    }
    pairs<EPV>(f, x);
}

// The kernel that adds the shares of dw and db is launched as the one before it ends, and
// waits for its writes (0.5 us sooner than an ordinary launch; started any earlier, it
// slowed the other by 1.3 us).
__device__ __forceinline__ void wait_for_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sums of N values over a team of lanes.
template <int N> __device__ __forceinline__ void lane_sum(float (&x)[N], int lanes) {
    for (int d = 1; d < lanes; d *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
}
// Over a team of whole warps: `threads` of them meet at barrier `bar`, once. red: [32][N],
// not used again before all of them have met at another barrier.
template <int N> __device__ __forceinline__ void warps_sum(float (&x)[N], int threads, int bar, float* red) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
    if (threads == 32) return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x % threads / 32;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[warp * N + i] = x[i];
    asm volatile("bar.sync %0, %1;" :: "r"(bar), "r"(threads) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = lane * 32 < threads ? red[lane * N + i] : 0.f;
#pragma unroll
    for (int d = 1; d < 32; d *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
}

// ---- rows of more than 32 vectors: a CTA a (row, group)
template <typename T, int EPV, int NV>
__global__ void __launch_bounds__(EPV == 1 && NV == 32 ? 1024 : kMaxTeam) layer_norm_fwd_kernel(NormArgs a) {
    __shared__ float red[2 * 32];
    const int64_t unit = blockIdx.x, row = a.groups == 1 ? unit : unit / a.groups;
    const int64_t c0 = (unit - row * a.groups) * a.width;
    const int t = threadIdx.x, team = blockDim.x;
    const T* x = static_cast<const T*>(a.x) + row * a.xs + c0;
    Raw<T, EPV> raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (t + v * team) * EPV;
        raw[v].zero();
        if (c < a.width) raw[v].load(x + c);
    }
    using P = Pk<EPV>;
    constexpr int N = kPk<EPV>;
    P f[NV][N], sum = both<P>(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        raw[v].widen(f[v]);
#pragma unroll
        for (int e = 0; e < N; ++e) sum = add2(sum, f[v][e]);
    }
    float s[1] = {total(sum)};
    warps_sum<1>(s, team, 0, red);
    const float mean = s[0] * a.inv_width;
    const P minus = both<P>(-mean);
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        P q = both<P>(0.f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            f[v][e] = add2(f[v][e], minus);
            q = fma2(f[v][e], f[v][e], q);
        }
        if ((t + v * team) * EPV < a.width) s[0] += total(q);
    }
    warps_sum<1>(s, team, 0, red + 32);
    const float rstd = rsqrtf(fmaf(s[0], a.inv_width, a.eps));
    if (t == 0 && a.mean) {
        a.mean[unit] = mean;
        a.rstd[unit] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ys + c0;
    const P scale = both<P>(rstd);
    auto finish = [&](auto type) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (t + v * team) * EPV;
            if (c < a.width) {
                P w[N], b[N];
                load_w<decltype(type), EPV>(a.w, c0 + c, 1.f, w);
                load_w<decltype(type), EPV>(a.b, c0 + c, 0.f, b);
#pragma unroll
                for (int e = 0; e < N; ++e) f[v][e] = fma2(mul2(f[v][e], scale), w[e], b[e]);
                store<T, EPV>(y + c, f[v]);
            }
        }
    };
    if (a.w_f32) finish(float());
    else finish(__nv_bfloat16());
}

// CTA blockIdx.x has rows blockIdx.x, + slots, ... of group blockIdx.y; its teams take
// them in turn. A thread copies its vectors of the rows ahead into shared memory of its
// own (no other thread reads them, so no barrier is needed): registers for one row
// alone are in use, and with rows loaded to registers HBM idled during each row's sums.
template <typename T, int EPV, int NV>
__global__ void __launch_bounds__(kMaxTeam, 1) layer_norm_bwd_kernel(NormArgs a) {
    constexpr int A = kAhead<EPV, NV>;
    extern __shared__ uint4 ahead[];             // [A][2][NV][threads]; at the end float [teams][2][width], their shares
    __shared__ float red[2][32 * 2];             // rows in turn
    const int team = a.team, t = threadIdx.x % team, me = threadIdx.x / team, teams = blockDim.x / team;
    const int grp = blockIdx.y;
    const int64_t c0 = (int64_t)grp * a.width, step = (int64_t)teams * a.slots;
    const T *x = static_cast<const T*>(a.x) + c0 + t * EPV, *dy = static_cast<const T*>(a.dy) + c0 + t * EPV;
    auto fetch = [&](int64_t row, int at) {      // the copies of one row are one group, be they none
        if constexpr (A > 0) {
            if (row < a.n) {
                const T *px = x + row * a.xs, *pd = dy + row * a.dys;
                uint4* dst = ahead + at * 2 * NV * blockDim.x + threadIdx.x;
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if ((t + v * team) * EPV < a.width) {
                        copy16(dst + v * blockDim.x, px + v * team * EPV);
                        copy16(dst + (NV + v) * blockDim.x, pd + v * team * EPV);
                    }
            }
            copies_commit();
        }
    };
    int64_t row = blockIdx.x + (int64_t)me * a.slots;
#pragma unroll
    for (int i = 0; i < A; ++i) fetch(row + i * step, i);
    // A row's statistics are on the way while the row before is worked on.
    float mean_next = row < a.n ? a.mean[row * a.groups + grp] : 0.f, rstd_next = row < a.n ? a.rstd[row * a.groups + grp] : 0.f;
    using P = Pk<EPV>;
    constexpr int N = kPk<EPV>;
    P w[NV][N], dw[NV][N], db[NV][N];
    auto weights = [&](auto type) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (t + v * team) * EPV;
            load_w<decltype(type), EPV>(c < a.width ? a.w : nullptr, c0 + c, 1.f, w[v]);
        }
    };
    if (a.w_f32) weights(float());
    else weights(__nv_bfloat16());
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[v][e] = db[v][e] = both<P>(0.f);
    int at = 0;
    for (int turn = 0; row < a.n; row += step, turn ^= 1) {
        Raw<T, EPV> rx[NV], rd[NV];
        if constexpr (A > 0) copies_wait<(A > 0 ? A - 1 : 0)>();
        const uint4* src = ahead + at * 2 * NV * blockDim.x + threadIdx.x;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            rx[v].zero();
            rd[v].zero();
            if ((t + v * team) * EPV < a.width) {
                if constexpr (A > 0) {
                    rx[v].u = src[v * blockDim.x];
                    rd[v].u = src[(NV + v) * blockDim.x];
                } else {
                    rx[v].load(x + row * a.xs + v * team * EPV);
                    rd[v].load(dy + row * a.dys + v * team * EPV);
                }
            }
        }
        fetch(row + A * step, at);
        at = at + 1 >= A ? 0 : at + 1;
        const float mean = mean_next, rstd = rstd_next;
        if (row + step < a.n) {
            mean_next = a.mean[(row + step) * a.groups + grp];
            rstd_next = a.rstd[(row + step) * a.groups + grp];
        }
        const P minus = both<P>(-mean), scale = both<P>(rstd);
        P s0 = both<P>(0.f), s1 = s0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {           // (behind the group's columns dy is zero)
            P f[N], d[N];
            rx[v].widen(f);
            rd[v].widen(d);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const P h = mul2(add2(f[e], minus), scale), u = mul2(d[e], w[v][e]);
                dw[v][e] = fma2(d[e], h, dw[v][e]);
                db[v][e] = add2(db[v][e], d[e]);
                s0 = add2(s0, u);
                s1 = fma2(u, h, s1);
            }
        }
        if (!a.dx) continue;
        float s[2] = {total(s0), total(s1)};
        warps_sum<2>(s, team, 1 + me, red[turn] + me * (team / 32) * 2);
        const P m1 = both<P>(-s[0] * a.inv_width * rstd), m2 = both<P>(-s[1] * a.inv_width * rstd);
        T* dx = static_cast<T*>(a.dx) + row * a.dxs + c0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (t + v * team) * EPV;
            if (c < a.width) {
                P f[N], d[N];
                rx[v].widen(f);
                rd[v].widen(d);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    d[e] = fma2(mul2(add2(f[e], minus), scale), m2, fma2(mul2(d[e], w[v][e]), scale, m1));
                store<T, EPV>(dx + c, d);
            }
        }
    }
    if (!a.part) return;
    // The teams' shares, added in the order of the teams.
    const int64_t cols = (int64_t)a.groups * a.width;
    float *share = reinterpret_cast<float*>(ahead), *pw = a.part + blockIdx.x * 2 * cols + c0;
    if (teams > 1) __syncthreads();              // every team is through with its copies
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        float gw[EPV], gb[EPV];
        singles<EPV>(dw[v], gw);
        singles<EPV>(db[v], gb);
        const int c = (t + v * team) * EPV;
        if (c >= a.width) continue;
        float *ow = teams > 1 ? share + me * 2 * a.width + c : pw + c, *ob = teams > 1 ? ow + a.width : ow + cols;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            ow[e] = gw[e];
            ob[e] = gb[e];
        }
    }
    if (teams == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.width; c += blockDim.x) {
        float sum = share[c];
        for (int m = 1; m < teams; ++m) sum += share[m * 2 * a.width + c];
        pw[c < a.width ? c : cols + c - a.width] = sum;
    }
}

// ---- backward of rows too wide for a thread's registers: the columns' sums by themselves, then
// dx by a CTA a (row, group), which reads its row twice (the second time from L1 or L2). 2048
// rows of 16384 columns in bf16 93 us, with the kernel above and its spills 410; of 8191, by
// single elements, 80 and 596.
template <typename T, int EPV> __global__ void __launch_bounds__(kMaxTeam) layer_norm_wide_dx_kernel(NormArgs a) {
    __shared__ float red[2 * 32];
    const int64_t unit = blockIdx.x, row = a.groups == 1 ? unit : unit / a.groups, c0 = (unit - row * a.groups) * a.width;
    const T *x = static_cast<const T*>(a.x) + row * a.xs + c0, *dy = static_cast<const T*>(a.dy) + row * a.dys + c0;
    T* dx = static_cast<T*>(a.dx) + row * a.dxs + c0;
    const float mean = a.mean[unit], rstd = a.rstd[unit];
    using P = Pk<EPV>;
    constexpr int N = kPk<EPV>;
    const P minus = both<P>(-mean), scale = both<P>(rstd);
    auto run = [&](auto type) {
        P s0 = both<P>(0.f), s1 = s0;
#pragma unroll 4
        for (int c = threadIdx.x * EPV; c < a.width; c += kMaxTeam * EPV) {
            Raw<T, EPV> rx, rd;
            rx.load(x + c);
            rd.load(dy + c);
            P f[N], d[N], w[N];
            rx.widen(f);
            rd.widen(d);
            load_w<decltype(type), EPV>(a.w, c0 + c, 1.f, w);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const P u = mul2(d[e], w[e]);
                s0 = add2(s0, u);
                s1 = fma2(u, mul2(add2(f[e], minus), scale), s1);
            }
        }
        float s[2] = {total(s0), total(s1)};
        warps_sum<2>(s, kMaxTeam, 0, red);
        const P m1 = both<P>(-s[0] * a.inv_width * rstd), m2 = both<P>(-s[1] * a.inv_width * rstd);
#pragma unroll 4
        for (int c = threadIdx.x * EPV; c < a.width; c += kMaxTeam * EPV) {
            Raw<T, EPV> rx, rd;
            rx.load(x + c);
            rd.load(dy + c);
            P f[N], d[N], w[N];
            rx.widen(f);
            rd.widen(d);
            load_w<decltype(type), EPV>(a.w, c0 + c, 1.f, w);
#pragma unroll
            for (int e = 0; e < N; ++e)
                d[e] = fma2(mul2(add2(f[e], minus), scale), m2, fma2(mul2(d[e], w[e]), scale, m1));
            store<T, EPV>(dx + c, d);
        }
    };
    if (a.w_f32) run(float());
    else run(__nv_bfloat16());
}

// A thread has EPV columns (all groups' laid end to end) of rows blockIdx.y, + slots, ...
template <typename T, int EPV> __global__ void __launch_bounds__(kThreads) layer_norm_wide_cols_kernel(NormArgs a) {
    const int64_t cols = (int64_t)a.groups * a.width, c = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * EPV;
    if (c >= cols) return;
    const int grp = (int)(c / a.width);
    using P = Pk<EPV>;
    constexpr int N = kPk<EPV>;
    P dw[N], db[N];
#pragma unroll
    for (int e = 0; e < N; ++e) dw[e] = db[e] = both<P>(0.f);
    const T *x = static_cast<const T*>(a.x) + c, *dy = static_cast<const T*>(a.dy) + c;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < a.n; row += a.slots) {
        Raw<T, EPV> rx, rd;
        rx.load(x + row * a.xs);
        rd.load(dy + row * a.dys);
        const P minus = both<P>(-a.mean[row * a.groups + grp]), scale = both<P>(a.rstd[row * a.groups + grp]);
        P f[N], d[N];
        rx.widen(f);
        rd.widen(d);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            dw[e] = fma2(d[e], mul2(add2(f[e], minus), scale), dw[e]);
            db[e] = add2(db[e], d[e]);
        }
    }
    float gw[EPV], gb[EPV], *pw = a.part + blockIdx.y * 2 * cols + c;
    singles<EPV>(dw, gw);
    singles<EPV>(db, gb);
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
        pw[e] = gw[e];
        pw[cols + e] = gb[e];
    }
}

// ---- groups of up to 32 vectors: teams of lanes, numbered so that neighbours take
// neighbouring groups of one row; a team has rows slot, slot + slots, ..., kBatch of
// them at a time, to have their loads on the way together
struct LaneTeam {
    int t, grp;
    int64_t slot, c0, rounds;
    __device__ __forceinline__ explicit LaneTeam(const NormArgs& a) {
        const int64_t id = (int64_t)blockIdx.x * (kThreads / a.team) + threadIdx.x / a.team;
        t = threadIdx.x % a.team;
        slot = a.groups == 1 ? id : id / a.groups;
        grp = (int)(id - slot * a.groups);
        c0 = (int64_t)grp * a.width;
        // Every team of a warp makes the same number of rounds: its lanes meet in the sums.
        rounds = (a.n + (int64_t)a.slots * kBatch - 1) / ((int64_t)a.slots * kBatch);
    }
};

// (CTAs an SM, by registers: 4096 rows of 28 groups of 128 took 17.6 us with two instead of 12.0, backward 44 with one)
template <typename T, int EPV> __global__ void __launch_bounds__(kThreads, 3) layer_norm_lanes_fwd_kernel(NormArgs a) {
    const LaneTeam k(a);
    const int c = k.t * EPV;
    const bool mine = c < a.width && k.slot < a.slots;
    using P = Pk<EPV>;
    constexpr int N = kPk<EPV>;
    P w[N], b[N];
    auto weights = [&](auto type) {
        load_w<decltype(type), EPV>(mine ? a.w : nullptr, k.c0 + c, 1.f, w);
        load_w<decltype(type), EPV>(mine ? a.b : nullptr, k.c0 + c, 0.f, b);
    };
    for (int64_t it = 0; it < k.rounds; ++it) {
        Raw<T, EPV> raw[kBatch];
        float mean[kBatch], rstd[kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int64_t row = (it * kBatch + r) * a.slots + k.slot;
            raw[r].zero();
            if (mine && row < a.n) raw[r].load(static_cast<const T*>(a.x) + row * a.xs + k.c0 + c);
        }
        if (it == 0) {                           // (behind the first rows' loads)
            if (a.w_f32) weights(float());
            else weights(__nv_bfloat16());
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            P f[N], q = both<P>(0.f);
            raw[r].widen(f);
#pragma unroll
            for (int e = 0; e < N; ++e) q = add2(q, f[e]);
            mean[r] = total(q);
        }
        lane_sum<kBatch>(mean, a.team);
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            P f[N], q = both<P>(0.f);
            raw[r].widen(f);
            mean[r] *= a.inv_width;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const P d = add2(f[e], both<P>(-mean[r]));
                q = fma2(d, d, q);
            }
            rstd[r] = mine ? total(q) : 0.f;
        }
        lane_sum<kBatch>(rstd, a.team);
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int64_t row = (it * kBatch + r) * a.slots + k.slot;
            if (!mine || row >= a.n) continue;
            rstd[r] = rsqrtf(fmaf(rstd[r], a.inv_width, a.eps));
            if (k.t == 0 && a.mean) {
                a.mean[row * a.groups + k.grp] = mean[r];
                a.rstd[row * a.groups + k.grp] = rstd[r];
            }
            P f[N];
            raw[r].widen(f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = fma2(mul2(add2(f[e], both<P>(-mean[r])), both<P>(rstd[r])), w[e], b[e]);
            store<T, EPV>(static_cast<T*>(a.y) + row * a.ys + k.c0 + c, f);
        }
    }
}

template <typename T, int EPV> __global__ void __launch_bounds__(kThreads, 2) layer_norm_lanes_bwd_kernel(NormArgs a) {
    const LaneTeam k(a);
    const int c = k.t * EPV;
    const bool mine = c < a.width && k.slot < a.slots;
    using P = Pk<EPV>;
    constexpr int N = kPk<EPV>;
    P w[N], dw[N], db[N];
    auto weights = [&](auto type) { load_w<decltype(type), EPV>(mine ? a.w : nullptr, k.c0 + c, 1.f, w); };
#pragma unroll
    for (int e = 0; e < N; ++e) dw[e] = db[e] = both<P>(0.f);
    for (int64_t it = 0; it < k.rounds; ++it) {
        Raw<T, EPV> rx[kBatch], rd[kBatch];
        float mean[kBatch], rstd[kBatch], s[2 * kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int64_t row = (it * kBatch + r) * a.slots + k.slot;
            rx[r].zero();
            rd[r].zero();
            mean[r] = rstd[r] = 0.f;
            if (mine && row < a.n) {
                rx[r].load(static_cast<const T*>(a.x) + row * a.xs + k.c0 + c);
                rd[r].load(static_cast<const T*>(a.dy) + row * a.dys + k.c0 + c);
                mean[r] = a.mean[row * a.groups + k.grp];
                rstd[r] = a.rstd[row * a.groups + k.grp];
            }
        }
        if (it == 0) {                           // (behind the first rows' loads)
            if (a.w_f32) weights(float());
            else weights(__nv_bfloat16());
        }
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            P f[N], d[N], s0 = both<P>(0.f), s1 = s0;
            rx[r].widen(f);
            rd[r].widen(d);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const P h = mul2(add2(f[e], both<P>(-mean[r])), both<P>(rstd[r])), u = mul2(d[e], w[e]);
                dw[e] = fma2(d[e], h, dw[e]);
                db[e] = add2(db[e], d[e]);
                s0 = add2(s0, u);
                s1 = fma2(u, h, s1);
            }
            s[2 * r] = total(s0);
            s[2 * r + 1] = total(s1);
        }
        if (!a.dx) continue;
        lane_sum<2 * kBatch>(s, a.team);
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int64_t row = (it * kBatch + r) * a.slots + k.slot;
            if (!mine || row >= a.n) continue;
            const P m1 = both<P>(-s[2 * r] * a.inv_width * rstd[r]), m2 = both<P>(-s[2 * r + 1] * a.inv_width * rstd[r]);
            P f[N], d[N];
            rx[r].widen(f);
            rd[r].widen(d);
#pragma unroll
            for (int e = 0; e < N; ++e)
                d[e] = fma2(mul2(add2(f[e], both<P>(-mean[r])), both<P>(rstd[r])), m2, fma2(mul2(d[e], w[e]), both<P>(rstd[r]), m1));
            store<T, EPV>(static_cast<T*>(a.dx) + row * a.dxs + k.c0 + c, d);
        }
    }
    if (!a.part || !mine) return;
    const int64_t cols = (int64_t)a.groups * a.width;
    float* pw = a.part + k.slot * 2 * cols + k.c0 + c;
    float gw[EPV], gb[EPV];
    singles<EPV>(dw, gw);
    singles<EPV>(db, gb);
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
        pw[e] = gw[e];
        pw[cols + e] = gb[e];
    }
}

// dw and db from the slots' shares: 32 columns a CTA, 8 runs of slots, added in order.
__global__ void __launch_bounds__(256) layer_norm_sum_kernel(NormArgs a) {
    __shared__ float red[8][33];
    wait_for_kernels();
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

// Vectors of a thread and threads of a team (lanes of a warp, or whole warps) for groups of nvec vectors.
struct Shape {
    int nv, team;
    bool lanes;
};
Shape shape_for(int64_t nvec, int usual, int most, int threads) {
    int t = 1, nv = usual;
    if (nvec <= 32) {
        while (t < nvec) t *= 2;
        return {1, t, true};
    }
    while (nv < most && nvec > threads * (int64_t)nv) nv *= 2;
    return {nv, (int)((nvec + 32 * nv - 1) / (32 * nv) * 32), false};
}
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
// Of groups of `width` columns, read by vectors or by single elements.
template <typename T> Shape shape_of(int64_t width, bool vec, bool bwd) {
    if (!vec) return shape_for(width, 8, 32, kMaxTeam);
    return bwd ? shape_for(width / kVec<T>, 2, 32 / kVec<T>, kMaxTeam) : shape_for(width / kVec<T>, 4, 16, kMaxTeam);
}

// Lane teams, or CTAs, that share a group's rows. Lane teams: what the GPU holds at once and
// no more (4096 rows of 28 heads of 128 columns, backward: 23.7 us, with a few CTAs above it
// 33). CTAs, of which an SM holds one: for each group the SMs' share rounded up, which is more
// than all hold at once where the groups do not divide 152 (28 groups: 168 CTAs, a second
// wave of 16). 152 is a constant, as the scratch's size must not depend on the current
// device. But four rows each at least (64 rows of 3584 columns: 10.0 us, with eight 11.9; two were no
// faster), and in the backward 608 lane teams at most, as every share of dw and db is
// written and read again (8192 rows of 128 columns: 16.3 us; with 2048 teams 21.7).
int slots_of(int64_t n, int groups, const Shape& sh, bool bwd) {
    const int64_t all = sh.lanes ? 152 * (bwd ? 2 : 3) * (kThreads / sh.team) / groups : (152 + groups - 1) / groups;
    return (int)std::max<int64_t>(1, std::min({(n + 3) / 4, all, int64_t(bwd && sh.lanes ? 608 : 1 << 30)}));
}

template <typename T, int EPV, int NV> cudaError_t run(NormArgs& a, bool bwd, cudaStream_t s) {
    ProfScope ps(bwd ? "layer_norm_bwd_kernel" : "layer_norm_fwd_kernel", s);
    if constexpr (NV >= 4) {                     // (shape_of)
        if (!bwd) {
            if (a.n * a.groups > kMaxGrid) return cudaErrorInvalidConfiguration;
            layer_norm_fwd_kernel<T, EPV, NV><<<(unsigned)(a.n * a.groups), a.team, 0, s>>>(a);
            return cudaGetLastError();
        }
    }
    if constexpr (NV * EPV <= 16) {              // (wider ones: run_wide)
        const int teams = std::max(1, kMaxTeam / a.team), threads = teams * a.team;
        const size_t copies = (size_t)kAhead<EPV, NV> * 2 * NV * threads * 16;
        const size_t smem = std::max(copies, teams > 1 && a.part ? teams * 2 * a.width * sizeof(float) : 0);
        static SmemGrant grant;
        const cudaError_t e = allow_smem(layer_norm_bwd_kernel<T, EPV, NV>, smem, grant);
        if (e != cudaSuccess) return e;
        layer_norm_bwd_kernel<T, EPV, NV><<<dim3(a.slots, a.groups), threads, smem, s>>>(a);
    }
    return cudaGetLastError();
}

// The columns first: dx may be dy itself, which they read.
template <typename T, int EPV> cudaError_t run_wide(NormArgs& a, cudaStream_t s) {
    if (a.dx && a.n * a.groups > kMaxGrid) return cudaErrorInvalidConfiguration;
    if (a.part) {
        ProfScope ps("layer_norm_wide_cols_kernel", s);
        const int64_t tiles = ((int64_t)a.groups * a.width / EPV + kThreads - 1) / kThreads;
        layer_norm_wide_cols_kernel<T, EPV><<<dim3((unsigned)tiles, a.slots), kThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!a.dx) return cudaSuccess;
    ProfScope ps("layer_norm_wide_dx_kernel", s);
    layer_norm_wide_dx_kernel<T, EPV><<<(unsigned)(a.n * a.groups), kMaxTeam, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int EPV> cudaError_t run_lanes(NormArgs& a, bool bwd, cudaStream_t s) {
    const int64_t units = (int64_t)a.slots * a.groups, grid = (units + kThreads / a.team - 1) / (kThreads / a.team);
    if (grid > kMaxGrid) return cudaErrorInvalidConfiguration;
    ProfScope ps(bwd ? "layer_norm_lanes_bwd_kernel" : "layer_norm_lanes_fwd_kernel", s);
    if (bwd) layer_norm_lanes_bwd_kernel<T, EPV><<<(unsigned)grid, kThreads, 0, s>>>(a);
    else layer_norm_lanes_fwd_kernel<T, EPV><<<(unsigned)grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch(NormArgs& a, bool bwd, bool vec, cudaStream_t s) {
    const Shape sh = shape_of<T>(a.width, vec, bwd);
    a.team = sh.team;
    a.slots = slots_of(a.n, a.groups, sh, bwd);
    a.inv_width = 1.f / (float)a.width;
    if (sh.lanes) return vec ? run_lanes<T, kVec<T>>(a, bwd, s) : run_lanes<T, 1>(a, bwd, s);
    if (bwd && (vec ? sh.nv * kVec<T> > 16 : sh.nv > 8)) return vec ? run_wide<T, kVec<T>>(a, s) : run_wide<T, 1>(a, s);
    if (!vec) return sh.nv == 8 ? run<T, 1, 8>(a, bwd, s) : run<T, 1, 32>(a, bwd, s);
    if (sh.nv == 2) return run<T, kVec<T>, 2>(a, bwd, s);
    if (sh.nv == 4) return run<T, kVec<T>, 4>(a, bwd, s);
    if (sh.nv == 8) return run<T, kVec<T>, 8>(a, bwd, s);
    return run<T, kVec<T>, 16>(a, bwd, s);
}

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

pkv_status norm_args(const pkv_norm* norm, int64_t n, NormArgs* a, const char* who) {
    const std::string w(who);
    if (!norm) return fail(PKV_ERR_INVALID, w + ": norm is NULL");
    if ((norm->dtype != PKV_BF16 && norm->dtype != PKV_F32) || (norm->w_dtype != PKV_BF16 && norm->w_dtype != PKV_F32))
        return fail(PKV_ERR_INVALID, w + ": dtype and w_dtype must be PKV_BF16 or PKV_F32");
    if (norm->groups > 65535) return fail(PKV_ERR_UNSUPPORTED, w + ": at most 65535 groups");
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

int slots_for(const pkv_norm* norm, int64_t n, bool vec) {
    const Shape sh = norm->dtype == PKV_BF16 ? shape_of<__nv_bfloat16>(norm->width, vec, true) : shape_of<float>(norm->width, vec, true);
    return slots_of(n, norm->groups, sh, true);
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
        const cudaError_t e = norm->dtype == PKV_BF16 ? launch<__nv_bfloat16>(a, false, vec, cs) : launch<float>(a, false, vec, cs);
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
            if (!dx && !a.part) return PKV_OK;
            const cudaError_t e = norm->dtype == PKV_BF16 ? launch<__nv_bfloat16>(a, true, vec, cs) : launch<float>(a, true, vec, cs);
            if (e != cudaSuccess) return cuda_fail(e, "pkv_layer_norm_bwd: launch");
        }
        if (!dw && !db) return PKV_OK;
        // (no rows: dw and db are sums of nothing)
        ProfScope ps("layer_norm_sum_kernel", cs);
        const int64_t cols = norm->groups * norm->width;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)((cols + 31) / 32), 2); cfg.blockDim = dim3(256); cfg.stream = cs;
        cfg.attrs = &attr; cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, layer_norm_sum_kernel, a);
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_layer_norm_bwd: launch");
    });
}

}  // extern "C"
