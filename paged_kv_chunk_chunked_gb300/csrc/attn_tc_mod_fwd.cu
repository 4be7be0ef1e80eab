// Tensor-core (tcgen05) attention forward with modified scores (mod.cuh), bf16
// in, fp32 accumulate: a query chunk against its pages.
//
// A CTA runs two streams, each a tile of 128 query rows of one head, over the
// same K and V pages of one KV head: two heads of a group, or a head of the next
// query tile where the group's number is odd. While the softmax warps of one
// stream work on its scores, the tensor core computes the other's products, so
// neither waits for the other's latency. (One stream per CTA with its rows'
// halves on two warpgroups in step left the tensor core idle for the length of
// each softmax: 28 heads, d 128, 4096 queries on 16384 keys took 665 us, 985 us
// with a cap, against 562 us, 774 us: 0.80 and 0.58 of the measured bf16 rate.
// What bounds it now: with a cap the fp32 pipe and the two warps a scheduler has
// to hide latency with (tensor pipe 40% active, fp32 pipe 38%, issue slots 48%);
// and about 13 us a CTA of start-up, masked first tile and epilogue.)
//   warps 0..3    softmax of stream 0, thread = query row, all 128 keys of a tile
//   warps 4..7    softmax of stream 1
//   warp 8        TMA: both Q tiles, then K and V pages into rings
//   warp 9        MMA issuer; order: PV0(j), S0(j+1), PV1(j), S1(j+1)
// S (fp32, 128 columns of tensor memory a stream) is overwritten by P (bf16, its
// first 64), P by the next S; tensor memory is full (2 x 128 + 2 x D columns), so
// Q stays in shared memory, where the A operand costs the tensor core a third
// more per instruction. O is rescaled in tensor memory only when a row's maximum
// grows by more than 2^8; S(j) complete says that PV(j-1) is, so no wait of its
// own stands before that. Weights are rounded to bf16 for the product (what the tensor
// core takes); their sum l comes from the unrounded ones, so that the LSE, which the
// backward forms P from, is fp32's. O is divided by the same l: where values share a
// large common part it is off by the mean rounding of its row's weights, up to 2^-8 of
// that part, which the plain kernel, dividing by the rounded weights' sum, is not; the
// plain LSE carries that rounding instead. (Both sums would cost four more operations
// a pair of keys in a loop that the softmax bounds.)
// Pages are walked from the last to the first: the distance bias lets the maximum
// grow towards the query's own position, and each growth costs a rescaling.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mod.cuh"
#include "tc.cuh"

namespace pkv {
namespace {

using tc::drain_wait;

constexpr int kTile = 128;                   // query rows = keys per tile
constexpr int kThreads = 320;
constexpr uint32_t kHalfBytes = 128 * 128;   // [128 rows][64 bf16] = 16 KB
constexpr int kKStages = 2, kVStages = 2;
constexpr float kRescaleThreshold = 8.0f;    // log2 units
constexpr float kBiasSlack = 64.0f;          // log2 units, of fp32's 126 below 1
constexpr int kShort = 1, kLong = 2, kAny = 3;   // forms of tanh

template <int D> struct Layout {
    static_assert(D == 64 || D == 128, "head dim 64 or 128");
    static constexpr int kBlocks = D / 64;                     // 64-column blocks
    static constexpr uint32_t kTileBytes = kBlocks * kHalfBytes;
    static constexpr uint32_t kOffQ = 0;                       // 2 streams
    static constexpr uint32_t kOffK = kOffQ + 2 * kTileBytes;
    static constexpr uint32_t kOffV = kOffK + kKStages * kTileBytes;
    static constexpr uint32_t kSmemBytes = kOffV + kVStages * kTileBytes + 1024;   // + alignment slack
};

struct Params {
    int Hq, Hkv;
    int per_tile;                    // streams of a query tile: the group's heads, padded to even with a selection
    int64_t q_start, n_q;
    void* o;
    float* lse;
    const int32_t* bt;
    int64_t num_phys;
    const int32_t* sel;
    int kmax;
    int* err;
    ModArgs m;
    float* part;                     // keys split over gridDim.y CTAs: partial results (attn_part_floats), else null
};

struct __align__(8) Barriers {
    uint64_t q_full;
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t s_full[2], p_full[2];   // per stream
    uint64_t o_full[2];
    uint64_t drain;
    uint32_t tmem_base;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
fwd_mod_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v, Params p) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Barriers B;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int kvh = (int)(blockIdx.x % p.Hkv), pair = (int)(blockIdx.x / p.Hkv), g = p.Hq / p.Hkv;
    const int n_qt = (int)((p.n_q + kTile - 1) / kTile);
    // Stream s: longest query tiles first; an odd one out repeats the other (`live` false).
    int qt[2], head[2];
    bool live[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int idx = 2 * pair + s;
        const int back = idx / p.per_tile, hh = idx - back * p.per_tile;
        live[s] = back < n_qt && hh < g;
        qt[s] = live[s] ? n_qt - 1 - back : qt[0];
        head[s] = live[s] ? kvh * g + hh : head[0];
    }
    // Pages: those the two tiles' ranges touch, or the selection's (one query tile then).
    const int32_t* sel_row = p.sel ? p.sel + ((size_t)qt[0] * p.Hkv + kvh) * p.kmax : nullptr;
    TileRange tr[2];
    tr[0] = tile_range<kTile>(p.m, p.q_start, (int64_t)qt[0] * kTile, p.n_q, lane);
    tr[1] = qt[1] == qt[0] ? tr[0] : tile_range<kTile>(p.m, p.q_start, (int64_t)qt[1] * kTile, p.n_q, lane);
    int first, nt;                           // tile j is entry first - j of the page list (dense: that page)
    {
        const int lo = tr[0].hi == 0 ? tr[1].lo : tr[1].hi == 0 ? tr[0].lo : min(tr[0].lo, tr[1].lo);
        const int hi = max(tr[0].hi, tr[1].hi);
        const int p0 = sel_row ? 0 : lo / kTile;
        const int n = sel_row ? sel_count_warp(sel_row, p.kmax, lane) : (hi + kTile - 1) / kTile - p0;
        const int s0 = (int)((int64_t)n * blockIdx.y / gridDim.y), s1 = (int)((int64_t)n * (blockIdx.y + 1) / gridDim.y);
        nt = s1 - s0;
        first = p0 + s1 - 1;
    }
    if (threadIdx.x == 0) {
        tc::mbar_init(&B.q_full, 1);
        for (int s = 0; s < kKStages; ++s) {
            tc::mbar_init(&B.k_full[s], 1);
            tc::mbar_init(&B.k_empty[s], 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            tc::mbar_init(&B.v_full[s], 1);
            tc::mbar_init(&B.v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&B.s_full[s], 1);
            tc::mbar_init(&B.p_full[s], 128);
            tc::mbar_init(&B.o_full[s], 1);
        }
        tc::mbar_init(&B.drain, 1);
        tc::fence_barrier_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(&B.tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = B.tmem_base;       // S0 [0, 128), S1 [128, 256), O0 [256, 256 + D), O1 [256 + D, 256 + 2 D)

    if (warp == 8) {
        // ------------------------------------------------------------ TMA producer
        tc::PageBatch pages;
        pages.init(p.bt, sel_row, nt, lane, first, -1, (int)((p.m.n_keys + kTile - 1) / kTile));
        if (lane == 0) {
            tc::prefetch_tmap(&tmap_k);
            tc::prefetch_tmap(&tmap_v);
            tc::mbar_arrive_expect_tx(&B.q_full, 2 * L::kTileBytes);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < L::kBlocks; ++b)
                    tc::tma_load_3d(smem + L::kOffQ + s * L::kTileBytes + b * kHalfBytes, &tmap_q, &B.q_full, 64 * b, head[s],
                                    qt[s] * kTile);
        }
        int k_issued = 0, v_issued = 0;
        for (int j = 0; j < nt; ++j) {
            const int ks = j % kKStages, vs = j % kVStages;
            if (j >= kKStages && !tc::warp_wait(&B.k_empty[ks], ((j / kKStages) - 1) & 1, p.err)) break;
            const int32_t pp = pages.get(j);
            int row = (int)(((int64_t)pp * p.Hkv + kvh) * kTile);
            if (pp < 0 || pp >= p.num_phys) {
                // Fine where neither tile sees the page: all its keys are masked, and
                // the rows before the first of the pool read as zero.
                const int64_t lp = sel_row ? sel_row[first - j] : first - j, k0 = lp * kTile;
                if (k0 >= p.m.n_keys ||
                    tile_sees<kTile>(p.m, p.q_start, (int64_t)qt[0] * kTile, p.n_q, (int)k0, (int)k0 + kTile) ||
                    tile_sees<kTile>(p.m, p.q_start, (int64_t)qt[1] * kTile, p.n_q, (int)k0, (int)k0 + kTile)) {
                    if (lane == 0) report_error(p.err, kErrBadPage);
                    break;
                }
                row = -kTile;
            }
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&B.k_full[ks], L::kTileBytes);
#pragma unroll
                for (int b = 0; b < L::kBlocks; ++b)
                    tc::tma_load_2d(smem + L::kOffK + ks * L::kTileBytes + b * kHalfBytes, &tmap_k, &B.k_full[ks], 64 * b, row);
            }
            k_issued = j + 1;
            if (j >= kVStages && !tc::warp_wait(&B.v_empty[vs], ((j / kVStages) - 1) & 1, p.err)) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&B.v_full[vs], L::kTileBytes);
#pragma unroll
                for (int b = 0; b < L::kBlocks; ++b)
                    tc::tma_load_2d(smem + L::kOffV + vs * L::kTileBytes + b * kHalfBytes, &tmap_v, &B.v_full[vs], 64 * b, row);
            }
            v_issued = j + 1;
        }
        // None of this CTA's copies may still be landing when it exits.
        if (lane == 0) {
            drain_wait(&B.q_full, 0);
            for (int j = max(0, k_issued - kKStages); j < k_issued; ++j) drain_wait(&B.k_full[j % kKStages], (j / kKStages) & 1);
            for (int j = max(0, v_issued - kVStages); j < v_issued; ++j) drain_wait(&B.v_full[j % kVStages], (j / kVStages) & 1);
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------ MMA issuer
        // The whole warp runs the loop (warp-uniform descriptors); one elected
        // lane issues the tcgen05 instructions and commits.
        const bool leader = tc::elect_one_sync();
        const uint32_t id_s = tc::idesc_bf16(128, 128, false, false);       // S = Q K^T
        const uint32_t id_pv = tc::idesc_bf16(128, D, false, true);         // O += P V
        const uint64_t dq0 = tc::sdesc(tc::smem_u32(smem + L::kOffQ), 16, 1024);             // K-major
        const uint64_t dk0 = tc::sdesc(tc::smem_u32(smem + L::kOffK), 16, 1024);
        const uint64_t dv0 = tc::sdesc(tc::smem_u32(smem + L::kOffV), kHalfBytes, 1024);     // MN-major
        auto issue_s = [&](int s, int j) {
            tc::tc_fence_after();
            if (leader) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
                    tc::mma_bf16(tmem + s * 128, tc::sdesc_at(dq0, s * L::kTileBytes + off),
                                 tc::sdesc_at(dk0, (j % kKStages) * L::kTileBytes + off), id_s, kk > 0 ? 1u : 0u);
                }
                tc::mma_commit(&B.s_full[s]);
                if (s == 1) tc::mma_commit(&B.k_empty[j % kKStages]);
            }
            __syncwarp();
        };
        bool ok = tc::warp_wait(&B.q_full, 0, p.err);
        if (ok && nt > 0) {
            ok = tc::warp_wait(&B.k_full[0], 0, p.err);
            if (ok) {
                issue_s(0, 0);
                issue_s(1, 0);
            }
        }
        for (int j = 0; ok && j < nt; ++j) {
            const int vs = j % kVStages;
            if (j + 1 < nt) ok = tc::warp_wait(&B.k_full[(j + 1) % kKStages], ((j + 1) / kKStages) & 1, p.err);
            if (ok) ok = tc::warp_wait(&B.v_full[vs], (j / kVStages) & 1, p.err);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (ok) ok = tc::warp_wait(&B.p_full[s], j & 1, p.err);
                if (!ok) break;
                tc::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)       // 16 keys each: 8 columns of P, 2 row groups of V
                        tc::mma_bf16_ts(tmem + 256 + s * D, tmem + s * 128 + kk * 8,
                                        tc::sdesc_at(dv0, vs * L::kTileBytes + kk * 2048), id_pv, (j > 0 || kk > 0) ? 1u : 0u);
                    if (j + 1 == nt) tc::mma_commit(&B.o_full[s]);
                    if (s == 1) tc::mma_commit(&B.v_empty[vs]);
                }
                __syncwarp();
                if (j + 1 < nt) issue_s(s, j + 1);
            }
        }
        // Drain: nothing of ours may still run on the tensor core at exit.
        if (leader) {
            tc::mma_commit(&B.drain);
            drain_wait(&B.drain, 0);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int s = warp >> 2, quad = warp & 3;            // stream; TMEM lane quadrant
        const int row = quad * 32 + lane;
        const int my_qt = s ? qt[1] : qt[0], h = s ? head[1] : head[0];
        const TileRange t = s ? tr[1] : tr[0];
        const uint32_t t_s = tmem + s * 128 + ((uint32_t)(quad * 32) << 16);
        const uint32_t t_o = tmem + 256 + s * D + ((uint32_t)(quad * 32) << 16);
        const int64_t q_local = (int64_t)my_qt * kTile + row;
        const bool valid = (s ? live[1] : live[0]) && q_local < p.n_q;
        const int2 range = q_local < p.n_q ? row_range(p.m, p.q_start, q_local) : make_int2(0, 0);
        const int qtile = (int)(p.q_start + (int64_t)my_qt * kTile), qpos = qtile + row;
        const bool capped = p.m.cap > 0.f, biased = p.m.slopes != nullptr;
        const float sl2 = rsqrtf((float)D) * kLog2e;
        const float ms = capped || biased ? 1.f : sl2;       // scores are in units of 1 / ms log2
        const float slope2 = biased ? p.m.slopes[h] * kLog2e : 0.f;
        float m = -INFINITY, lsum = 0.f;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.s_full[s], j & 1, p.err));
            if (!ok) break;
            tc::tc_fence_after();
            const int kb = (sel_row ? sel_row[first - j] : first - j) * kTile;       // first key
            const float dist = (float)(kb - qpos);
            const bool mask = kb < t.full_lo || kb + kTile > t.full_hi;
            const int side = kb + kTile - 1 <= qtile ? -1 : kb >= qtile + kTile - 1 ? 1 : 0;

            // The row's new maximum (log2 units): O and l follow where it grows beyond the
            // threshold. PV(j - 1) is complete, and PV(j) waits for this row.
            auto grow = [&](float mx) {
                const bool up = mx > m + kRescaleThreshold;
                if (__any_sync(0xffffffffu, up)) {
                    const float f = !up ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - mx);
                    if (up) m = mx;
                    lsum *= f;
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t r[32];
                            tc::tmem_ld32(t_o + c * 32, r);
                            tc::tmem_wait_ld(r);
#pragma unroll
                            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                            tc::tmem_st32(t_o + c * 32, r);
                        }
                    }
                }
            };
            // The row is read twice, 32 keys at a time and the next 32 on their way: once for
            // the maximum, once for the weights. That keeps 64 scores in registers where all
            // 128 would spill, and the other stream fills the reads' latency.
            // (`again`: another reading follows, whose first load starts here.)
            uint32_t ra[32], rb[32];
            tc::tmem_ld32(t_s, ra);
            auto each_chunk = [&](auto again, auto&& use) {
#pragma unroll 1
                for (int c0 = 0; c0 < kTile; c0 += 64) {
                    tc::tmem_wait_ld(ra);
                    tc::tmem_ld32(t_s + c0 + 32, rb);
                    use(ra, c0);
                    tc::tmem_wait_ld(rb);
                    if (decltype(again)::value || c0 == 0) tc::tmem_ld32(t_s + (c0 == 0 ? 64 : 0), ra);
                    use(rb, c0 + 32);
                }
            };
            const std::true_type more{};
            const std::false_type last{};
            float neg_m = 0.f, sum[4] = {0.f, 0.f, 0.f, 0.f};
            // Weights of 32 keys into P, whose columns lie over keys that have been read by
            // then. late(emit) hands over the keys' scores, in units of 1 / ms.
            auto weights = [&](int c0, auto&& late) {
                uint32_t pk[16];
                late([&](int c, float x0, float x1) {
                    const float a = fast_exp2(fmaf(x0, ms, neg_m)), b = fast_exp2(fmaf(x1, ms, neg_m));
                    sum[c & 2] += a;
                    sum[(c & 2) + 1] += b;
                    pk[c >> 1] = pack_bf16x2(a, b);
                });
                tc::tmem_st16(t_s + c0 / 2, pk);
            };
            auto plain = [](const uint32_t (&r)[32], auto&& emit) {
#pragma unroll
                for (int c = 0; c < 32; c += 2) emit(c, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
            };
            auto pairs = [](auto&& emit) {
                return [&](int c, f32x2 y) {
                    float a, b;
                    unpack2(y, a, b);
                    emit(c, a, b);
                };
            };
            auto most = [](const uint32_t (&r)[32], float (&mp)[4]) {
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    mp[(c >> 1) & 3] = max3(mp[(c >> 1) & 3], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
            };
            float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto start = [&](float top) {
                grow(top);
                // (A row that has seen nothing yet keeps m = -inf; its weights are 0.)
                neg_m = m == -INFINITY ? 0.f : -m;
            };
            // Cap, bias and mask compiled in. CAP: 0, or the form of tanh; BIAS: 0, the side
            // of a tile that lies wholly before the queries (-1), or 1: any side.
            auto hide = [&](uint32_t (&r)[32], int c0) {
                const int lo = range.x - kb - c0, hi = range.y - kb - c0;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (c < lo || c >= hi) r[c] = 0xff800000u;
            };
            auto capped_pairs = [&](const uint32_t (&r)[32], auto form, auto&& use) {
                if constexpr (decltype(form)::value == kShort) cap_short(r, p.m, use);
                else if constexpr (decltype(form)::value == kLong) cap_long(r, p.m, use);
                else cap_any(r, p.m, use);
            };
            auto biased_pairs = [&](const uint32_t (&r)[32], float pre, int c0, auto kind, auto&& use) {
                bias_pairs(r, pre, slope2, dist + (float)c0, 1.f, decltype(kind)::value == -1 ? -1 : 0, use);
            };
            auto run = [&](auto cap_, auto bias_, auto mask_) {
                constexpr int CAP = decltype(cap_)::value, BIAS = decltype(bias_)::value;
                constexpr bool MASK = decltype(mask_)::value;
                // Scores of 32 keys from their raw logits, in place.
                auto scores = [&](uint32_t (&r)[32], int c0) {
                    if constexpr (CAP != 0) capped_pairs(r, cap_, [&](int c, f32x2 y) { put_pair(r, c, y); });
                    if constexpr (BIAS != 0)
                        biased_pairs(r, CAP != 0 ? 1.f : sl2, c0, bias_, [&](int c, f32x2 y) { put_pair(r, c, y); });
                    if constexpr (MASK) hide(r, c0);
                };
                if (CAP == 0 && BIAS == -1 && slope2 >= 0.f && slope2 * (kTile - 1) <= kBiasSlack) {
                    // The largest logit with the nearest key's bias bounds the maximum from
                    // above by at most the bias's span over the tile. The weights are floats:
                    // a reference 2^64 too high costs them nothing, and the tile's biases are
                    // formed once instead of twice.
                    each_chunk(more, [&](uint32_t (&r)[32], int) { most(r, mp); });
                    start(fmaf(fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]), sl2, slope2 * (dist + (kTile - 1))));
                } else if constexpr (CAP == 0 || BIAS != 0) {
                    each_chunk(more, [&](uint32_t (&r)[32], int c0) {
                        scores(r, c0);
                        most(r, mp);
                    });
                    start(fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]) * ms);
                } else {
                    // The capped maximum of the raw logits (which the caller has taken, for
                    // the form: of all the tile's keys, hidden ones too, unless MASK).
                    const float top = fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]);
                    start(top == -INFINITY ? top : p.m.c2 * tanh_any(top * p.m.k));
                }
                each_chunk(last, [&](uint32_t (&r)[32], int c0) {
                    if constexpr (MASK || (CAP != 0 && BIAS != 0)) {
                        scores(r, c0);
                        weights(c0, [&](auto&& emit) { plain(r, emit); });
                    } else if constexpr (CAP != 0) {
                        // (The cap's products go with the exponentials, on another pipe.)
                        weights(c0, [&](auto&& emit) { capped_pairs(r, cap_, pairs(emit)); });
                    } else if constexpr (BIAS != 0) {
                        weights(c0, [&](auto&& emit) { biased_pairs(r, sl2, c0, bias_, pairs(emit)); });
                    } else {
                        weights(c0, [&](auto&& emit) { plain(r, emit); });
                    }
                });
            };
            using std::integral_constant;
            const integral_constant<int, 0> no{};
            const integral_constant<int, -1> before{};
            const integral_constant<int, 1> any_side{};
            const integral_constant<bool, false> whole{};
            const integral_constant<bool, true> parts{};
            const integral_constant<int, kShort> short_form{};
            const integral_constant<int, kLong> long_form{};
            const integral_constant<int, kAny> any_form{};
            // Each kind of tile has its code to itself: a step that is skipped at run time
            // inside a common one still costs a move of its registers.
            if (!capped) {
                if (!biased) mask ? run(no, no, parts) : run(no, no, whole);
                else if (mask || side != -1) run(no, any_side, parts);
                else run(no, before, whole);
            } else {
                // The cap's form goes by the largest logit of the warp's rows.
                float top = 0.f;
                each_chunk(more, [&](uint32_t (&r)[32], int c0) {
                    top = fmaxf(top, abs_max(r));
                    if (mask) hide(r, c0);
                    most(r, mp);
                });
                top = warp_top(top) * p.m.k;
                if (!biased) {
                    if (mask) top <= kTanhShort ? run(short_form, no, parts) : run(any_form, no, parts);
                    else if (top <= kTanhShort) run(short_form, no, whole);
                    else if (top <= kTanhLong) run(long_form, no, whole);
                    else run(any_form, no, whole);
                } else {
                    mp[0] = mp[1] = mp[2] = mp[3] = -INFINITY;
                    if (top <= kTanhShort) {
                        if (mask || side != -1) run(short_form, any_side, parts);
                        else run(short_form, before, whole);
                    } else {
                        run(any_form, any_side, parts);
                    }
                }
            }
            lsum += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc::tmem_wait_st();
            tc::tc_fence_before();
            tc::mbar_arrive(&B.p_full[s]);
        }
        if (ok && nt > 0) ok = __all_sync(0xffffffffu, tc::mbar_wait(&B.o_full[s], 0, p.err));
        if (ok) {
            tc::tc_fence_after();
            const float inv = lsum == 0.f ? 0.f : 1.f / lsum;            // a row that saw nothing: O = 0
            const float lse2 = lsum == 0.f ? -INFINITY : m + log2f(lsum);
            const size_t hrow = (size_t)h * p.n_q + q_local;
            const size_t prow = (size_t)blockIdx.y * p.Hq * p.n_q + hrow;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                if (nt > 0) {
                    tc::tmem_ld32(t_o + c * 32, r);
                    tc::tmem_wait_ld(r);
                }
                if (!valid) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = lsum == 0.f ? 0u : __float_as_uint(__uint_as_float(r[e]) * inv);
                if (p.part) {
                    float4* dst = reinterpret_cast<float4*>(p.part + prow * D + c * 32);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dst[v] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                             __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
                } else {
                    __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o) + ((size_t)q_local * p.Hq + h) * D;
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint4*>(orow + c * 32 + v * 8) = make_uint4(
                            pack_bf16x2(__uint_as_float(r[8 * v]), __uint_as_float(r[8 * v + 1])),
                            pack_bf16x2(__uint_as_float(r[8 * v + 2]), __uint_as_float(r[8 * v + 3])),
                            pack_bf16x2(__uint_as_float(r[8 * v + 4]), __uint_as_float(r[8 * v + 5])),
                            pack_bf16x2(__uint_as_float(r[8 * v + 6]), __uint_as_float(r[8 * v + 7])));
                }
            }
            if (valid) {
                if (p.part) p.part[(size_t)gridDim.y * p.Hq * p.n_q * D + prow] = lse2;
                else p.lse[hrow] = lse2 * kLn2;
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    constexpr uint32_t smem = Layout<D>::kSmemBytes;
    static SmemGrant allowed;
    const cudaError_t e = allow_smem(fwd_mod_tc_kernel<D>, smem, allowed);
    if (e != cudaSuccess) return e;
    CUtensorMap tq;
    std::string why;
    if (!make_tmap_3d(&tq, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, a.Hq, a.n_q, (uint64_t)D * 2, (uint64_t)a.Hq * D * 2, 64, 1,
                      kTile, &why))
        return cudaErrorInvalidValue;
    Params p{};
    p.Hq = a.Hq; p.Hkv = a.Hkv; p.q_start = a.q_start; p.n_q = a.n_q;
    p.o = a.o; p.lse = a.lse; p.bt = a.bt; p.num_phys = a.num_phys;
    p.sel = a.sel; p.kmax = a.kmax; p.err = a.err; p.m = a.m;
    p.part = a.splits > 1 ? a.part : nullptr;
    const int g = a.Hq / a.Hkv;
    p.per_tile = a.sel ? (g + 1) / 2 * 2 : g;
    const int64_t streams = (a.n_q + kTile - 1) / kTile * p.per_tile;
    ProfScope ps("fwd_mod_tc_kernel", s);
    const dim3 grid((unsigned)((streams + 1) / 2 * a.Hkv), a.splits);
    fwd_mod_tc_kernel<D><<<grid, kThreads, smem, s>>>(tq, *a.tmap_k, *a.tmap_v, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_fwd_mod_tc(const AttnArgs& a, cudaStream_t s) {
    return a.d == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

// Few query tiles against a long cache leave most SMs idle: split the keys so
// that about two CTAs per SM run, each with at least 4 pages of its own.
int attn_fwd_mod_tc_splits(const AttnArgs& a) {
    if (a.sel) return 1;
    const int sms = sm_count();
    const int64_t streams = (a.n_q + kTile - 1) / kTile * (a.Hq / a.Hkv);
    const int64_t ctas = (streams + 1) / 2 * a.Hkv, pages = (a.m.n_keys + kTile - 1) / kTile;
    if (2 * ctas > sms) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({pages / 4, 2 * (int64_t)sms / ctas, 64}));
}

}  // namespace pkv
