// C entry points of the attention with modified scores (mod.cuh): argument
// checks, scratch and dispatch. Short bf16 calls go to the kernel for few
// queries; the tensor-core kernels take what they take of the plain calls (bf16,
// pages of 128 tokens, d 64 or 128), the CUDA-core kernels the rest.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "mod.cuh"

namespace pkv {
namespace {

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

// Fills a for a call with modified scores; *empty: there is nothing to do.
pkv_status mod_common(pkv_seq* s, const void* q, int64_t q_start, int64_t n_q, const pkv_score_mod* mod,
                      const pkv_sel* sel, AttnArgs* a, bool* empty, const char* who) {
    const std::string w(who);
    if (!s) return fail(PKV_ERR_INVALID, w + ": seq is NULL");
    if (!mod) return fail(PKV_ERR_INVALID, w + ": mod is NULL");
    if (!(mod->softcap == 0.f || (mod->softcap >= 1e-3f && mod->softcap <= 1e4f)))
        return fail(PKV_ERR_INVALID, w + ": softcap must be 0 (none) or in [1e-3, 1e4]");
    if (misaligned(mod->slopes, 4) || misaligned(mod->k_begin, 8) || misaligned(mod->k_end, 8))
        return fail(PKV_ERR_INVALID, w + ": slopes, k_begin or k_end is misaligned");
    if (q_start < 0 || n_q < 0 || q_start > s->len || n_q > s->len - q_start)
        return fail(PKV_ERR_INVALID, w + ": need 0 <= q_start and q_start + n_q <= length");
    if (sel && q_start % s->pool->desc.page_size)
        return fail(PKV_ERR_INVALID, w + ": with a selection q_start must be a multiple of the page size");
    *empty = n_q == 0;
    if (*empty) return PKV_OK;
    if (misaligned(q, 16)) return fail(PKV_ERR_INVALID, w + ": q must be 16-byte aligned");
    const pkv_status st = attn_common(s, q, q_start, n_q, sel, a, who, true);
    if (st != PKV_OK) return st;
    a->mod = true;
    a->m.k_begin = mod->k_begin;
    a->m.k_end = mod->k_end;
    a->m.slopes = mod->slopes;
    set_cap(&a->m, mod->softcap, s->pool->desc.head_dim);
    a->m.n_keys = mod->k_end ? s->len : q_start + n_q;
    a->splits = 1;
    return PKV_OK;
}

// Scratch of the sequence's calls, at least `floats` long. A larger buffer is
// allocated on demand; the smaller ones live on with the sequence, since a
// captured graph may hold their addresses.
pkv_status seq_scratch(pkv_seq* s, size_t floats, cudaStream_t cs, float** out, const char* who) {
    if (s->scratch_floats < floats) {
        if (capturing(cs))
            return fail(PKV_ERR_INVALID, std::string(who) + ": needs a larger scratch buffer than the sequence has; run the "
                                                            "call once before capturing it");
        const size_t want = std::max(floats, 2 * s->scratch_floats);
        s->retired.reserve(s->retired.size() + 1);
        float* p = nullptr;
        const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&p), want * sizeof(float));
        if (e != cudaSuccess) {
            cudaGetLastError();                        // the failure is reported, not left for the next launch check
            return cuda_fail(e, (std::string(who) + ": scratch").c_str());
        }
        if (s->scratch) s->retired.push_back(s->scratch);
        s->scratch = p;
        s->scratch_floats = want;
    }
    *out = s->scratch;
    return PKV_OK;
}

}  // namespace

bool capturing(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &st) == cudaSuccess) return st != cudaStreamCaptureStatusNone;
    cudaGetLastError();                                // the legacy stream while another one captures
    return true;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_chunk_attn_mod_fwd(pkv_seq* s, const void* q, int64_t q_start, int64_t n_q, void* o, float* lse,
                                  const pkv_score_mod* mod, const pkv_sel* sel, void* stream) {
    static const char* who = "pkv_chunk_attn_mod_fwd";
    return guarded(who, [&]() -> pkv_status {
        AttnArgs a{};
        bool empty = false;
        pkv_status st = mod_common(s, q, q_start, n_q, mod, sel, &a, &empty, who);
        if (st != PKV_OK || empty) return st;
        if (!o || !lse) return fail(PKV_ERR_INVALID, std::string(who) + ": o or lse is NULL");
        if (misaligned(o, 16) || misaligned(lse, 4))
            return fail(PKV_ERR_INVALID, std::string(who) + ": o must be 16-byte aligned, lse 4-byte aligned");
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if (s->used && capturing(cs))
            return fail(PKV_ERR_INVALID, std::string(who) + ": calls on a PINNED_HOST pool cannot be captured");
        a.o = o;
        a.lse = lse;
        const bool few = !(s->pool->desc.flags & PKV_FLAG_SIMT_ONLY) && few_supported(a), tc = use_tc(s->pool, a);
        a.splits = few ? attn_few_splits(a) : tc ? attn_fwd_mod_tc_splits(a) : attn_fwd_mod_simt_splits(a);
        if (a.splits > 1) {
            st = seq_scratch(s, attn_part_floats(a), cs, &a.part, who);
            if (st != PKV_OK) return st;
        }
        cudaError_t e = few ? launch_attn_few(a, cs) : tc ? launch_attn_fwd_mod_tc(a, cs) : launch_attn_fwd_mod_simt(a, cs);
        if (e == cudaSuccess && a.splits > 1) e = launch_attn_join(a, cs);
        if (e == cudaSuccess && s->used) e = cudaEventRecord(s->used, cs);
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_chunk_attn_mod_fwd: launch");
    });
}

pkv_status pkv_chunk_attn_mod_bwd(pkv_seq* s, const void* q, const void* o, const void* dout, const float* lse,
                                  int64_t q_start, int64_t n_q, void* dq, const pkv_score_mod* mod, const pkv_sel* sel,
                                  void* stream) {
    static const char* who = "pkv_chunk_attn_mod_bwd";
    return guarded(who, [&]() -> pkv_status {
        AttnArgs a{};
        bool empty = false;
        pkv_status st = mod_common(s, q, q_start, n_q, mod, sel, &a, &empty, who);
        if (st != PKV_OK || empty) return st;
        if (!o || !dout || !lse || !dq)
            return fail(PKV_ERR_INVALID, std::string(who) + ": o, dout, lse or dq is NULL");
        if (misaligned(o, 16) || misaligned(dout, 16) || misaligned(dq, 16) || misaligned(lse, 4))
            return fail(PKV_ERR_INVALID, std::string(who) + ": o, dout and dq must be 16-byte aligned, lse 4-byte aligned");
        if (s->pool->desc.page_size % 16)
            return fail(PKV_ERR_UNSUPPORTED, std::string(who) + ": the page size must be a multiple of 16");
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if (s->used && capturing(cs))
            return fail(PKV_ERR_INVALID, std::string(who) + ": calls on a PINNED_HOST pool cannot be captured");
        // Scratch: the bounds of the 64-query tiles, the queries' ranges, D [Hq * n_q]
        // and, with a selection, the page list and the query-page masks (8-byte aligned).
        const size_t n_b = 4 * (size_t)((n_q + 63) / 64) + 2 * (size_t)n_q, n_d = (size_t)a.Hq * n_q;
        const size_t n_list = sel ? 1 + (size_t)bwd_pagelist_cap(a) : 0;
        const size_t n_mask = sel ? 1 + 2 * (size_t)bwd_selmask_words(a) : 0;
        float* scratch = nullptr;
        st = seq_scratch(s, n_b + n_d + n_list + n_mask, cs, &scratch, who);
        if (st != PKV_OK) return st;
        a.o_in = o; a.dout = dout; a.lse_in = lse; a.dq = dq;
        a.bounds = reinterpret_cast<int4*>(scratch);
        a.ranges = reinterpret_cast<int2*>(scratch + 4 * (size_t)((n_q + 63) / 64));
        a.Dbuf = scratch + n_b;
        a.pagelist = sel ? reinterpret_cast<int32_t*>(a.Dbuf + n_d) : nullptr;
        a.selmask = sel ? reinterpret_cast<uint64_t*>(
                              (reinterpret_cast<uintptr_t>(a.Dbuf + n_d + n_list) + 7) & ~uintptr_t(7))
                        : nullptr;
        cudaError_t e;
        if (use_tc(s->pool, a)) {
            e = launch_attn_bwd_tc(a, cs);
        } else {
            e = launch_bwd_rowdot(a, cs);
            if (e == cudaSuccess) e = launch_attn_bwd_mod_simt(a, cs);
        }
        if (e == cudaSuccess && s->used) e = cudaEventRecord(s->used, cs);
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_chunk_attn_mod_bwd: launch");
    });
}

}  // extern "C"
