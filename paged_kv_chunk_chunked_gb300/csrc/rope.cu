// Position rotation of Q and K rows on their way into the paged cache, and the
// rotation back of their gradients on the way out.
//
// A pair (x, y) of a row at position p turns by the angle p * f, f the pair's
// frequency: (x, y) -> (x cos - y sin, y cos + x sin); the gradient of the
// turned pair turns by the opposite angle. Pairs are dims (i, i + r/2)
// (halves) or (2i, 2i + 1) (interleaved), i < r/2; dims from r on pass through.
//
// Angles: an fp32 product p * f is off by 2^-24 of the angle, 0.06 rad at one
// million radians, and the fp64 units are too few to form one product per
// (token, pair). So f is turned once per CTA into a 64-bit fixed-point
// fraction of a turn, rounded to nearest, and p * f is an integer product modulo
// 2^64: whole turns drop out by themselves and the phase is off by at most
// |p| * 2^-65 turns: 1.9e-7 rad at |p| = 2^40, 1.9e-4 at 2^50. Its leading 32 bits
// give cos and sin in fp32.
//
// The kernels are HBM-bound copies. A thread owns two 16-byte vectors of a row
// (slot v of SL = D / (2 * EPV)): in the rotated part the two vectors whose
// elements pair up (halves: vectors v and v + r/2/EPV; interleaved: 2v and
// 2v + 1), behind it two plain ones. Its EPV (cos, sin) pairs stay in
// registers for the heads it walks.
#include <cuda_bf16.h>

#include <algorithm>
#include <new>

#include "common.cuh"
#include "internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;       // 4096 tokens, 28/4 heads, d 128: append 20.6 us, gradient 16.6 us (256: 22.4, 18.0)
constexpr int kHeadGroup = 4;       // query heads per thread: 8 loads in flight, cos/sin computed once per 4
constexpr int kZeroSplit = 4;       // CTAs that zero one (page, KV head) gradient tile pair

struct RopeArgs {
    const float* inv_freq;
    const int64_t* positions;       // or null: pos0 + row
    int64_t pos0;
    int half;                       // rotated pairs per row
    bool interleaved;
};

// Fraction of a turn per position, as a 64-bit fixed-point number modulo one
// turn: f / (2 pi) * 2^64 from f's 24-bit mantissa times floor(2^96 / (2 pi)).
__device__ __forceinline__ uint64_t turns_fixed(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int ex = (bits >> 23) & 0xff;
    const uint32_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    // m * K, K = 0x28be60db 9391054a 7f09d5f4 (94 bits), as three 40-bit limbs' sum.
    const uint64_t p0 = (uint64_t)m * 0x7f09d5f4u, p1 = (uint64_t)m * 0x9391054au, p2 = (uint64_t)m * 0x28be60dbu;
    const uint64_t lo = p0 + (p1 << 32);
    const uint64_t hi = p2 + (p1 >> 32) + (lo < p0 ? 1u : 0u);
    // value * 2^64 = (m * K) / 2^s, s = 182 - ex, to nearest: the last bit shifted out rounds.
    const int s = 182 - max(ex, 1);
    uint64_t r = 0;
    if (s > 0) {
        const unsigned __int128 x = s <= 128 ? ((unsigned __int128)hi << 64 | lo) >> (s - 1) : 0;
        r = (uint64_t)(x >> 1) + ((uint64_t)x & 1u);
    } else if (s > -64) {
        r = lo << (-s);
    }
    return (bits >> 31) ? 0ull - r : r;
}

// Fills the CTA's table; whether a frequency is not finite, which no fraction of a turn is.
__device__ __forceinline__ bool fill_turns(uint64_t* fix, const RopeArgs& r) {
    bool bad = false;
    for (int i = threadIdx.x; i < r.half; i += blockDim.x) {
        const float f = r.inv_freq[i];
        bad |= !isfinite(f);
        fix[i] = turns_fixed(f);
    }
    return __syncthreads_or(bad);
}

// cos and sin of the N pairs from pair i0 on, at position pos (SIGN -1: of the
// opposite angle). bad: fill_turns'.
template <int N, int SIGN>
__device__ __forceinline__ void cos_sin(const uint64_t* fix, const RopeArgs& r, bool bad, int i0, int64_t pos, float (&c)[N],
                                        float (&s)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint64_t phase = (uint64_t)pos * fix[i0 + e];
        // Signed leading half: [-1/2, 1/2) turn; in half turns for sincospif.
        float t = (float)(int32_t)(phase >> 32) * (1.0f / 2147483648.0f);
        if (bad && !isfinite(r.inv_freq[i0 + e])) t = __uint_as_float(0x7fc00000u);      // NaN, as p * f would give
        sincospif(t, &s[e], &c[e]);
        if (SIGN < 0) s[e] = -s[e];
    }
}

template <int N>
__device__ __forceinline__ void turn(float (&a)[N], float (&b)[N], const float (&c)[N], const float (&s)[N],
                                     bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1];
            a[2 * e] = x * c[e] - y * s[e];
            a[2 * e + 1] = y * c[e] + x * s[e];
            const float u = b[2 * e], w = b[2 * e + 1];
            b[2 * e] = u * c[N / 2 + e] - w * s[N / 2 + e];
            b[2 * e + 1] = w * c[N / 2 + e] + u * s[N / 2 + e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float x = a[e], y = b[e];
            a[e] = x * c[e] - y * s[e];
            b[e] = y * c[e] + x * s[e];
        }
    }
}

// EPV floats -> one 16-byte vector of T (one rounding to nearest for bf16).
template <typename T> __device__ __forceinline__ uint4 narrow16(const float* f);
template <> __device__ __forceinline__ uint4 narrow16<float>(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 narrow16<__nv_bfloat16>(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// The two vectors of slot v.
template <typename T>
__device__ __forceinline__ void slot_vectors(int v, const RopeArgs& r, int& va, int& vb) {
    constexpr int EPV = 16 / (int)sizeof(T);
    const int hv = r.half / EPV;                  // slots that rotate
    if (v >= hv || r.interleaved) {
        va = 2 * v;
        vb = va + 1;
    } else {
        va = v;
        vb = v + hv;
    }
}

struct RowsArgs {
    const void* x;
    void* out;
    int64_t x_stride, out_stride;   // elements between rows
    int64_t n;
    int H;
};

// Rows of a [n, H, D] tensor rotated: thread (token, group of heads, slot). The
// CTA's angle table is filled while the rows' loads are on their way.
template <typename T, int D, int SIGN>
__device__ __forceinline__ void rotate_rows(const RowsArgs& a, const RopeArgs& r, uint64_t* fix, int64_t unit) {
    constexpr int EPV = 16 / (int)sizeof(T), SL = D / (2 * EPV);
    const int v = (int)(unit % SL);
    const int groups = (a.H + kHeadGroup - 1) / kHeadGroup;
    const int64_t tg = unit / SL;
    const int64_t t = tg / groups;
    const int h0 = (int)(tg - t * groups) * kHeadGroup;
    int va, vb;
    slot_vectors<T>(v, r, va, vb);
    const bool rot = v < r.half / EPV;
    const T* src = static_cast<const T*>(a.x) + t * a.x_stride + (size_t)h0 * D;
    T* dst = static_cast<T*>(a.out) + t * a.out_stride + (size_t)h0 * D;
    const int nh = t < a.n ? min(kHeadGroup, a.H - h0) : 0;
    uint4 xa[kHeadGroup], xb[kHeadGroup];
#pragma unroll
    for (int h = 0; h < kHeadGroup; ++h)
        if (h < nh) {                              // plain loads: out may be x itself
            xa[h] = reinterpret_cast<const uint4*>(src + h * D)[va];
            xb[h] = reinterpret_cast<const uint4*>(src + h * D)[vb];
        }
    const int64_t pos = r.positions && nh > 0 ? r.positions[t] : r.pos0 + t;
    const bool bad = fill_turns(fix, r);
    if (rot && nh > 0) {
        float c[EPV], s[EPV];
        cos_sin<EPV, SIGN>(fix, r, bad, v * EPV, pos, c, s);
#pragma unroll
        for (int h = 0; h < kHeadGroup; ++h)
            if (h < nh) {
                float fa[EPV], fb[EPV];
                widen16<T>(xa[h], fa);
                widen16<T>(xb[h], fb);
                turn<EPV>(fa, fb, c, s, r.interleaved);
                xa[h] = narrow16<T>(fa);
                xb[h] = narrow16<T>(fb);
            }
    }
#pragma unroll
    for (int h = 0; h < kHeadGroup; ++h)
        if (h < nh) {
            reinterpret_cast<uint4*>(dst + h * D)[va] = xa[h];
            reinterpret_cast<uint4*>(dst + h * D)[vb] = xb[h];
        }
}

template <typename T, int D>
int64_t rows_units(const RowsArgs& a) {
    constexpr int EPV = 16 / (int)sizeof(T), SL = D / (2 * EPV);
    return a.n * ((a.H + kHeadGroup - 1) / kHeadGroup) * SL;
}

template <typename T, int D, int SIGN>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(RowsArgs a, RopeArgs r) {
    __shared__ uint64_t fix[D / 2];
    rotate_rows<T, D, SIGN>(a, r, fix, (int64_t)blockIdx.x * kThreads + threadIdx.x);
}

// ---------------------------------------------------------------- append

// CTAs [0, kv_ctas): one (logical page, KV head) each -- its new K rows
// rotated and its V rows copied into the page, and the page's representative;
// then zero_ctas that zero the gradient tiles of the pages this call starts;
// then the CTAs that rotate Q.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_rope_kernel(AppendArgs a, int64_t k_stride, int64_t v_stride,
                                                              RowsArgs q, RopeArgs r, int kv_ctas, int zero_ctas) {
    constexpr int EPV = 16 / (int)sizeof(T), SL = D / (2 * EPV);
    constexpr int RSTEP = kThreads / SL;
    __shared__ uint64_t fix[D / 2];
    __shared__ float red[RSTEP][D];
    static_assert(kThreads >= D, "one thread per dimension of the representative");
    const int P = a.P, tid = threadIdx.x;
    int b = (int)blockIdx.x;
    if (b >= kv_ctas + zero_ctas) {
        rotate_rows<T, D, 1>(q, r, fix, (int64_t)(b - kv_ctas - zero_ctas) * kThreads + tid);
        return;
    }
    const bool zero = b >= kv_ctas;
    int part = 0;
    if (zero) {
        b -= kv_ctas;
        part = b % kZeroSplit;
        b /= kZeroSplit;
    }
    const int h = b % a.Hkv;
    const int64_t lp = a.old_len / P + b / a.Hkv;
    const int64_t page_start = lp * P;
    const int32_t pp = a.bt[lp];
    if (pp < 0 || pp >= a.num_phys) {
        report_error(a.err, kErrBadPage);
        return;
    }
    const size_t page_off = ((size_t)pp * a.Hkv + h) * (size_t)P * D;
    if (zero) {
        // A page taken off the free list starts with zero gradient (for host
        // pages only recorded as such, nothing crosses the host link).
        if (page_start < a.old_len) return;
        if (a.gzero) {
            if (part == 0 && tid == 0) a.gzero[(size_t)pp * a.Hkv + h] = 1;
            return;
        }
        float4* g0 = reinterpret_cast<float4*>(a.dkpool + page_off);
        float4* g1 = reinterpret_cast<float4*>(a.dvpool + page_off);
        const int n4 = P * D / 4, from = n4 / kZeroSplit * part, to = part + 1 < kZeroSplit ? from + n4 / kZeroSplit : n4;
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = from + tid; i < to; i += kThreads) {
            g0[i] = z;
            g1[i] = z;
        }
        return;
    }
    const int v = tid % SL, r0 = tid / SL;
    int va, vb;
    slot_vectors<T>(v, r, va, vb);
    const bool rot = v < r.half / EPV;
    const int64_t new_len = a.old_len + a.n_tok;
    T* kpage = static_cast<T*>(a.kpool) + page_off;
    T* vpage = static_cast<T*>(a.vpool) + page_off;
    float acc_a[EPV], acc_b[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) acc_a[e] = acc_b[e] = 0.f;
    constexpr int U = 2;                          // rows in flight per thread
    bool table = false, bad = false;
    for (int rb0 = 0; rb0 < P; rb0 += U * RSTEP) {
        const int rb = rb0 + r0;
        uint4 ka[U], kb[U], wa[U], wb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = rb + u * RSTEP;
            const int64_t pos = page_start + row;
            ka[u] = kb[u] = wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
            if (row < P && pos >= a.old_len && pos < new_len) {
                const int64_t t = pos - a.old_len;
                const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_in) + t * k_stride + (size_t)h * D);
                const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_in) + t * v_stride + (size_t)h * D);
                ka[u] = __ldg(ks + va);
                kb[u] = __ldg(ks + vb);
                wa[u] = __ldg(vs + va);
                wb[u] = __ldg(vs + vb);
            } else if (row < P && pos < a.old_len) {
                ka[u] = reinterpret_cast<const uint4*>(kpage + (size_t)row * D)[va];   // stored by an earlier append
                kb[u] = reinterpret_cast<const uint4*>(kpage + (size_t)row * D)[vb];
            }
        }
        if (!table) bad = fill_turns(fix, r);           // while the first rows' loads are on their way
        table = true;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = rb + u * RSTEP;
            const int64_t pos = page_start + row;
            if (row >= P) continue;
            float fa[EPV], fb[EPV];
            if (pos >= a.old_len) {               // new rows, and zero rows beyond the sequence
                if (rot && pos < new_len) {
                    const int64_t t = pos - a.old_len;
                    float c[EPV], s[EPV];
                    cos_sin<EPV, 1>(fix, r, bad, v * EPV, r.positions ? r.positions[t] : r.pos0 + t, c, s);
                    widen16<T>(ka[u], fa);
                    widen16<T>(kb[u], fb);
                    turn<EPV>(fa, fb, c, s, r.interleaved);
                    ka[u] = narrow16<T>(fa);
                    kb[u] = narrow16<T>(fb);
                }
                uint4* kd = reinterpret_cast<uint4*>(kpage + (size_t)row * D);
                uint4* vd = reinterpret_cast<uint4*>(vpage + (size_t)row * D);
                kd[va] = ka[u];
                kd[vb] = kb[u];
                vd[va] = wa[u];
                vd[vb] = wb[u];
            }
            if (pos < new_len) {                  // the representative averages the keys as stored
                widen16<T>(ka[u], fa);
                widen16<T>(kb[u], fb);
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    acc_a[e] += fa[e];
                    acc_b[e] += fb[e];
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
        red[r0][va * EPV + e] = acc_a[e];
        red[r0][vb * EPV + e] = acc_b[e];
    }
    __syncthreads();
    if (tid < D) {
        float sum = 0.f;
#pragma unroll 8
        for (int g = 0; g < RSTEP; ++g) sum += red[g][tid];
        a.rep[((size_t)pp * a.Hkv + h) * D + tid] = sum / (float)min64(P, new_len - page_start);
    }
}

// ---------------------------------------------------------------- gradient

struct GradArgs {
    const float* dkpool;
    const float* dvpool;
    const uint8_t* gzero;           // PINNED_HOST: tiles recorded as zero (memory stale), or null
    const int32_t* bt;
    int64_t num_phys;
    int P, Hkv;
    int64_t row0, n;
    void* dk;
    void* dv;
    int64_t dk_stride, dv_stride;
    int* err;
};

// EPV floats of a gradient row from page memory.
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(p + e));
        f[e] = x.x; f[e + 1] = x.y; f[e + 2] = x.z; f[e + 3] = x.w;
    }
}

// CTAs [0, kv_ctas): thread (row, KV head, slot) turns the row's dK back,
// rounds it and dV once and writes both; the rest turn dQ back.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_grad_kernel(GradArgs a, RowsArgs q, RopeArgs r, int kv_ctas) {
    constexpr int EPV = 16 / (int)sizeof(T), SL = D / (2 * EPV);
    __shared__ uint64_t fix[D / 2];
    if ((int)blockIdx.x >= kv_ctas) {
        rotate_rows<T, D, -1>(q, r, fix, (int64_t)((int)blockIdx.x - kv_ctas) * kThreads + threadIdx.x);
        return;
    }
    const int64_t unit = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int v = (int)(unit % SL);
    const int64_t th = unit / SL;
    const int64_t t = th / a.Hkv;
    const int h = (int)(th - t * a.Hkv);
    const bool live = t < a.n;
    const int64_t row = a.row0 + (live ? t : 0), lp = row / a.P;
    const int32_t pp = a.bt[lp];
    const bool ok = live && pp >= 0 && pp < a.num_phys;
    if (live && !ok) report_error(a.err, kErrBadPage);
    int va, vb;
    slot_vectors<T>(v, r, va, vb);
    float fa[EPV], fb[EPV], ga[EPV], gb[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) fa[e] = fb[e] = ga[e] = gb[e] = 0.f;
    if (ok) {
        const size_t tile = (size_t)pp * a.Hkv + h;
        const size_t off = (tile * a.P + (size_t)(row - lp * a.P)) * D;
        if (!(a.gzero && a.gzero[tile])) {         // else recorded as zero, the memory is stale
            if (a.dk) {
                load_f32<EPV>(a.dkpool + off + va * EPV, fa);
                load_f32<EPV>(a.dkpool + off + vb * EPV, fb);
            }
            if (a.dv) {
                load_f32<EPV>(a.dvpool + off + va * EPV, ga);
                load_f32<EPV>(a.dvpool + off + vb * EPV, gb);
            }
        }
    }
    const int64_t pos = r.positions && live ? r.positions[t] : r.pos0 + t;
    const bool bad = fill_turns(fix, r);
    if (!ok) return;
    if (a.dk) {
        if (v < r.half / EPV) {
            float c[EPV], s[EPV];
            cos_sin<EPV, -1>(fix, r, bad, v * EPV, pos, c, s);
            turn<EPV>(fa, fb, c, s, r.interleaved);
        }
        uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(a.dk) + t * a.dk_stride + (size_t)h * D);
        d[va] = narrow16<T>(fa);
        d[vb] = narrow16<T>(fb);
    }
    if (a.dv) {
        uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(a.dv) + t * a.dv_stride + (size_t)h * D);
        d[va] = narrow16<T>(ga);
        d[vb] = narrow16<T>(gb);
    }
}

// ---------------------------------------------------------------- launches

constexpr int64_t kMaxRows = int64_t(1) << 31;      // a pool holds fewer rows than that
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

int64_t ctas(int64_t units) { return (units + kThreads - 1) / kThreads; }

template <typename T, int D>
cudaError_t launch_append_rope(const AppendArgs& a, int64_t ks, int64_t vs, const RowsArgs& q, const RopeArgs& r,
                               cudaStream_t s) {
    const int64_t pages = (a.old_len + a.n_tok - 1) / a.P - a.old_len / a.P + 1;
    const int64_t kv = pages * a.Hkv, zero = kv * kZeroSplit, nq = ctas(rows_units<T, D>(q));
    if (kv + zero + nq > kMaxGrid) return cudaErrorInvalidConfiguration;
    ProfScope ps("append_rope_kernel", s);
    append_rope_kernel<T, D><<<(unsigned)(kv + zero + nq), kThreads, 0, s>>>(a, ks, vs, q, r, (int)kv, (int)zero);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rope_rows(const RowsArgs& a, const RopeArgs& r, bool inverse, cudaStream_t s) {
    const int64_t n = ctas(rows_units<T, D>(a));
    if (n > kMaxGrid) return cudaErrorInvalidConfiguration;
    ProfScope ps("rope_rows_kernel", s);
    if (inverse) rope_rows_kernel<T, D, -1><<<(unsigned)n, kThreads, 0, s>>>(a, r);
    else rope_rows_kernel<T, D, 1><<<(unsigned)n, kThreads, 0, s>>>(a, r);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rope_grad(const GradArgs& a, const RowsArgs& q, const RopeArgs& r, cudaStream_t s) {
    constexpr int SL = D * (int)sizeof(T) / 32;
    const int64_t kv = a.dk || a.dv ? ctas(a.n * a.Hkv * SL) : 0;
    const int64_t nq = q.x ? ctas(rows_units<T, D>(q)) : 0;
    if (kv + nq > kMaxGrid) return cudaErrorInvalidConfiguration;
    if (kv + nq == 0) return cudaSuccess;
    ProfScope ps("rope_grad_kernel", s);
    rope_grad_kernel<T, D><<<(unsigned)(kv + nq), kThreads, 0, s>>>(a, q, r, (int)kv);
    return cudaGetLastError();
}

#define PKV_BY_TYPE(pool, call)                                                                   \
    ((pool)->desc.dtype == PKV_BF16                                                               \
         ? ((pool)->desc.head_dim == 128 ? call(__nv_bfloat16, 128) : call(__nv_bfloat16, 64))    \
         : ((pool)->desc.head_dim == 128 ? call(float, 128) : call(float, 64)))

// Checks the rotation and fills r.
pkv_status rope_args(const pkv_pool* p, const pkv_rope* rope, RopeArgs* r, const char* who) {
    if (!rope || !rope->inv_freq)
        return fail(PKV_ERR_INVALID, std::string(who) + ": rope or rope->inv_freq is NULL");
    if (rope->rotary_dim <= 0 || rope->rotary_dim > p->desc.head_dim || rope->rotary_dim % 2)
        return fail(PKV_ERR_INVALID, std::string(who) + ": rotary_dim must be even and in 2..head_dim");
    if (rope->rotary_dim % 16)
        return fail(PKV_ERR_UNSUPPORTED, std::string(who) + ": rotary_dim must be a multiple of 16");
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return fail(PKV_ERR_INVALID, std::string(who) + ": interleaved must be 0 or 1");
    if ((reinterpret_cast<uintptr_t>(rope->inv_freq) & 3) || (reinterpret_cast<uintptr_t>(rope->positions) & 7))
        return fail(PKV_ERR_INVALID, std::string(who) + ": inv_freq or positions is misaligned");
    r->inv_freq = rope->inv_freq;
    r->positions = rope->positions;
    r->pos0 = rope->pos0;
    r->half = rope->rotary_dim / 2;
    r->interleaved = rope->interleaved != 0;
    return PKV_OK;
}

// A [n, H, d] operand whose rows are `stride` elements apart (0: dense).
pkv_status rows_check(const pkv_pool* p, const void* x, int H, int64_t* stride, const char* who, const char* name) {
    const int64_t dense = (int64_t)H * p->desc.head_dim, epv = 16 / (int64_t)p->elem;
    if (*stride == 0) *stride = dense;
    if (*stride < dense || *stride % epv || (reinterpret_cast<uintptr_t>(x) & 15))
        return fail(PKV_ERR_INVALID, std::string(who) + ": " + name + " must be 16-byte aligned, with rows at least heads * " +
                                         "head_dim elements and a multiple of 16 bytes apart");
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_append_rope(pkv_seq* s, const void* q, int64_t q_stride, void* q_out, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, int64_t n_tok, const pkv_rope* rope, void* stream) {
    static const char* who = "pkv_append_rope";
    return guarded(who, [&]() -> pkv_status {
        if (!s || n_tok < 0) return fail(PKV_ERR_INVALID, "pkv_append_rope: bad argument");
        const pkv_pool* p = s->pool;
        RopeArgs r{};
        pkv_status st = rope_args(p, rope, &r, who);
        if (st != PKV_OK) return st;
        if (n_tok == 0) return PKV_OK;
        if (n_tok > kMaxRows) return fail(PKV_ERR_INVALID, "pkv_append_rope: n_tok out of range");
        if (!k || !v) return fail(PKV_ERR_INVALID, "pkv_append_rope: k or v is NULL");
        if (!q != !q_out) return fail(PKV_ERR_INVALID, "pkv_append_rope: q and q_out go together");
        RowsArgs qa{q, q_out, q_stride, 0, q ? n_tok : 0, p->desc.n_q_heads};
        if (q && (st = rows_check(p, q, qa.H, &qa.x_stride, who, "q")) != PKV_OK) return st;
        if (q && (st = rows_check(p, q_out, qa.H, &qa.out_stride, who, "q_out")) != PKV_OK) return st;
        if ((st = rows_check(p, k, p->desc.n_kv_heads, &k_stride, who, "k")) != PKV_OK) return st;
        if ((st = rows_check(p, v, p->desc.n_kv_heads, &v_stride, who, "v")) != PKV_OK) return st;
        if (!is_device(p)) return fail(PKV_ERR_INVALID, "pkv_append_rope: META pool holds no data");
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if (capturing(cs))
            return fail(PKV_ERR_INVALID, "pkv_append_rope: an append advances the sequence on the host and cannot be captured");
        AppendArgs a{};
        st = append_begin(s, n_tok, false, cs, &a, who);
        if (st != PKV_OK) return st;
        a.k_in = k;
        a.v_in = v;
#define PKV_CALL(T, D) launch_append_rope<T, D>(a, k_stride, v_stride, qa, r, cs)
        return append_end(s, n_tok, PKV_BY_TYPE(p, PKV_CALL), cs, who);
#undef PKV_CALL
    });
}

pkv_status pkv_rope_rows(const pkv_pool* p, const void* x, int64_t x_stride, void* out, int64_t out_stride, int64_t n,
                         int32_t n_heads, const pkv_rope* rope, int32_t inverse, void* stream) {
    static const char* who = "pkv_rope_rows";
    return guarded(who, [&]() -> pkv_status {
        if (!p || n < 0 || n > kMaxRows || n_heads <= 0 || n_heads > (1 << 20) || (inverse != 0 && inverse != 1))
            return fail(PKV_ERR_INVALID, "pkv_rope_rows: bad argument");
        RopeArgs r{};
        pkv_status st = rope_args(p, rope, &r, who);
        if (st != PKV_OK) return st;
        if (n == 0) return PKV_OK;
        if (!x || !out) return fail(PKV_ERR_INVALID, "pkv_rope_rows: x or out is NULL");
        RowsArgs a{x, out, x_stride, out_stride, n, n_heads};
        if ((st = rows_check(p, x, n_heads, &a.x_stride, who, "x")) != PKV_OK) return st;
        if ((st = rows_check(p, out, n_heads, &a.out_stride, who, "out")) != PKV_OK) return st;
        if (!is_device(p)) return fail(PKV_ERR_INVALID, "pkv_rope_rows: META pool");
        if ((st = check_stream_device(p)) != PKV_OK) return st;
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
#define PKV_CALL(T, D) launch_rope_rows<T, D>(a, r, inverse != 0, cs)
        const cudaError_t e = PKV_BY_TYPE(p, PKV_CALL);
#undef PKV_CALL
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_rope_rows: launch");
    });
}

pkv_status pkv_rope_grad(pkv_seq* s, int64_t row0, int64_t n_rows, const pkv_rope* rope, const void* dq, int64_t dq_stride,
                         void* dq_out, int64_t dq_out_stride, void* dk_out, int64_t dk_stride, void* dv_out,
                         int64_t dv_stride, void* stream) {
    static const char* who = "pkv_rope_grad";
    return guarded(who, [&]() -> pkv_status {
        if (!s) return fail(PKV_ERR_INVALID, "pkv_rope_grad: seq is NULL");
        const pkv_pool* p = s->pool;
        if (row0 < 0 || n_rows < 0 || row0 > s->len || n_rows > s->len - row0)
            return fail(PKV_ERR_INVALID, "pkv_rope_grad: need 0 <= row0 and row0 + n_rows <= length");
        RopeArgs r{};
        pkv_status st = rope_args(p, rope, &r, who);
        if (st != PKV_OK) return st;
        if (!dq != !dq_out) return fail(PKV_ERR_INVALID, "pkv_rope_grad: dq and dq_out go together");
        if (!is_device(p)) return fail(PKV_ERR_INVALID, "pkv_rope_grad: META pool");
        if (n_rows == 0 || (!dq && !dk_out && !dv_out)) return PKV_OK;
        RowsArgs qa{dq, dq_out, dq_stride, dq_out_stride, n_rows, p->desc.n_q_heads};
        GradArgs a{p->dk, p->dv, p->gzero, s->d_bt, p->desc.num_phys_pages, p->desc.page_size, p->desc.n_kv_heads,
                   row0, n_rows, dk_out, dv_out, dk_stride, dv_stride, p->d_err};
        if (dq && (st = rows_check(p, dq, qa.H, &qa.x_stride, who, "dq")) != PKV_OK) return st;
        if (dq && (st = rows_check(p, dq_out, qa.H, &qa.out_stride, who, "dq_out")) != PKV_OK) return st;
        if (dk_out && (st = rows_check(p, dk_out, a.Hkv, &a.dk_stride, who, "dk_out")) != PKV_OK) return st;
        if (dv_out && (st = rows_check(p, dv_out, a.Hkv, &a.dv_stride, who, "dv_out")) != PKV_OK) return st;
        if ((st = check_stream_device(p)) != PKV_OK) return st;
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
#define PKV_CALL(T, D) launch_rope_grad<T, D>(a, qa, r, cs)
        const cudaError_t e = PKV_BY_TYPE(p, PKV_CALL);
#undef PKV_CALL
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_rope_grad: launch");
    });
}

}  // extern "C"
