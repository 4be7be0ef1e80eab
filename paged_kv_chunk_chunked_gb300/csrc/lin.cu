// C entry points of linear attention (lin.cuh): the store of states, argument
// checks, scratch and dispatch.
#include <algorithm>

#include "lin.cuh"

namespace pkv {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;      // row numbers fit a TMA coordinate
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) & (to - 1); }

pkv_status operand(const pkv_lin* lin, const void* x, int H, int64_t stride, LinRows* out, const char* who, const char* name) {
    const int64_t dense = (int64_t)H * lin->desc.head_dim, epv = lin->desc.dtype == PKV_BF16 ? 8 : 4;
    if (stride == 0) stride = dense;
    if (!x) return fail(PKV_ERR_INVALID, std::string(who) + ": " + name + " is NULL");
    if (stride < dense || stride % epv || misaligned(x, 16))
        return fail(PKV_ERR_INVALID, std::string(who) + ": " + name + " must be 16-byte aligned, with rows at least heads * " +
                                         "head_dim elements and a multiple of 16 bytes apart");
    out->p = const_cast<void*>(x);
    out->stride = stride;
    return PKV_OK;
}

// Checks that need no operands, and fills a with the store's parts.
pkv_status begin(const pkv_lin* lin, int64_t n, const float* log_decay, LinArgs* a, const char* who) {
    const std::string w(who);
    if (!lin) return fail(PKV_ERR_INVALID, w + ": lin is NULL");
    if (n < 0 || n > kMaxRows) return fail(PKV_ERR_INVALID, w + ": n out of range");
    if (misaligned(log_decay, 4)) return fail(PKV_ERR_INVALID, w + ": log_decay is misaligned");
    a->Hq = lin->desc.n_q_heads; a->Hkv = lin->desc.n_kv_heads; a->d = lin->desc.head_dim; a->dtype = lin->desc.dtype;
    a->n = n; a->n_slots = lin->desc.n_slots;
    a->log_decay = log_decay;
    a->one_term = lin->desc.flags & PKV_FLAG_LIN_ONE_TERM;
    a->state = lin->state; a->dstate = lin->dstate; a->err = lin->d_err; a->wait_err = lin->d_err ? lin->d_err + 1 : nullptr;
    return PKV_OK;
}

pkv_status batch_args(const pkv_lin_batch* batch, LinArgs* a, const char* who) {
    const std::string w(who);
    if (!batch) return fail(PKV_ERR_INVALID, w + ": batch is NULL");
    if (batch->n_seq < 0 || batch->n_seq > kMaxRows || (!batch->cu && batch->n_seq != 1))
        return fail(PKV_ERR_INVALID, w + ": n_seq must be 1 without cu, and not negative");
    if (misaligned(batch->cu, 8) || misaligned(batch->slot_in, 4) || misaligned(batch->slot_out, 4))
        return fail(PKV_ERR_INVALID, w + ": cu, slot_in or slot_out is misaligned");
    a->n_seq = batch->n_seq;
    a->cu = batch->cu; a->slot_in = batch->slot_in; a->slot_out = batch->slot_out;
    const int64_t chunks = lin_chunks(a->n, a->n_seq, kLinSimtChunk);
    if (chunks > kMaxGrid / 2 || a->n_seq * a->Hkv > kMaxGrid / 64) return fail(PKV_ERR_UNSUPPORTED, w + ": too many sequences");
    return PKV_OK;
}

pkv_status on_device(const pkv_lin* lin, const char* who) {
    if (lin->desc.residency == PKV_RES_META) return fail(PKV_ERR_INVALID, std::string(who) + ": META store holds no states");
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev != lin->device)
        return fail(PKV_ERR_INVALID, std::string(who) + ": the current CUDA device is not the store's device");
    return PKV_OK;
}

// Whether the tensor-core kernels take the store's calls.
bool on_tensor_cores(const pkv_lin* lin) { return lin->desc.dtype == PKV_BF16 && !(lin->desc.flags & PKV_FLAG_SIMT_ONLY); }

// Scratch for the chunk states, of a backward also for their gradients.
pkv_status chunk_states(pkv_lin* lin, LinArgs* a, bool bwd, cudaStream_t cs, const char* who) {
    const bool tc = on_tensor_cores(lin);
    a->n_chunks = (int)lin_chunks(a->n, a->n_seq, tc ? kLinTcChunk : kLinSimtChunk);
    if ((int64_t)a->n_chunks * std::max(a->Hkv * a->d, a->Hkv + a->Hq) > kMaxGrid / 2) return fail(PKV_ERR_UNSUPPORTED, std::string(who) + ": too many rows");
    const size_t one = (size_t)a->n_chunks * a->Hkv * a->d * a->d, floats = one * (bwd ? 2 : 1);
    if (lin->scratch_floats < floats) {
        if (capturing(cs))
            return fail(PKV_ERR_INVALID, std::string(who) + ": needs a larger scratch buffer than the store has; run the call "
                                                            "once before capturing it");
        lin->retired.reserve(lin->retired.size() + 1);
        // At least twice the old buffer, so that all that were outgrown, which stay, are together
        // smaller than the new one; just what is needed where that is all there is room for.
        size_t size = std::max(floats, 2 * lin->scratch_floats);
        float* p = nullptr;
        cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&p), size * sizeof(float));
        if (e != cudaSuccess && size > floats) {
            cudaGetLastError();
            size = floats;
            e = cudaMalloc(reinterpret_cast<void**>(&p), size * sizeof(float));
        }
        if (e != cudaSuccess) {
            cudaGetLastError();                  // reported here, not left for the next launch check
            return cuda_fail(e, (std::string(who) + ": scratch").c_str());
        }
        if (lin->scratch) lin->retired.push_back(lin->scratch);
        lin->scratch = p;
        lin->scratch_floats = size;
    }
    a->part = lin->scratch;
    a->gpart = bwd ? lin->scratch + one : nullptr;
    return PKV_OK;
}

pkv_status launched(cudaError_t e, const std::string& why, const char* who) {
    if (e == cudaSuccess) return PKV_OK;
    return why.empty() ? cuda_fail(e, (std::string(who) + ": launch").c_str()) : fail(PKV_ERR_CUDA, std::string(who) + ": " + why);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_lin_create(const pkv_lin_desc* d, pkv_lin** out) {
    return guarded("pkv_lin_create", [&]() -> pkv_status {
        if (!out) return fail(PKV_ERR_INVALID, "pkv_lin_create: out is NULL");
        *out = nullptr;
        if (!d) return fail(PKV_ERR_INVALID, "pkv_lin_create: desc is NULL");
        if (d->n_kv_heads <= 0 || d->n_q_heads <= 0 || d->n_q_heads % d->n_kv_heads)
            return fail(PKV_ERR_INVALID, "pkv_lin_create: n_q_heads must be a positive multiple of n_kv_heads");
        if (d->n_q_heads > 65535) return fail(PKV_ERR_UNSUPPORTED, "pkv_lin_create: at most 65535 heads");
        if (d->head_dim != 64 && d->head_dim != 128)
            return fail(PKV_ERR_UNSUPPORTED, "pkv_lin_create: head_dim must be 64 or 128");
        if (d->dtype != PKV_BF16 && d->dtype != PKV_F32)
            return fail(PKV_ERR_INVALID, "pkv_lin_create: dtype must be PKV_BF16 or PKV_F32");
        if (d->residency != PKV_RES_DEVICE && d->residency != PKV_RES_META)
            return fail(PKV_ERR_INVALID, "pkv_lin_create: residency must be PKV_RES_DEVICE or PKV_RES_META");
        if (d->grads != 0 && d->grads != 1) return fail(PKV_ERR_INVALID, "pkv_lin_create: grads must be 0 or 1");
        if (d->n_slots <= 0 || d->n_slots > (int64_t(1) << 30))
            return fail(PKV_ERR_INVALID, "pkv_lin_create: n_slots must be in 1 .. 2^30");
        if (d->flags & ~(PKV_FLAG_SIMT_ONLY | PKV_FLAG_LIN_ONE_TERM)) return fail(PKV_ERR_INVALID, "pkv_lin_create: unknown flags");
        pkv_lin* lin = new pkv_lin();
        lin->desc = *d;
        if (d->residency == PKV_RES_META) {
            *out = lin;
            return PKV_OK;
        }
        const size_t bytes = (size_t)d->n_slots * d->n_kv_heads * d->head_dim * d->head_dim * sizeof(float);
        cudaError_t e = cudaGetDevice(&lin->device);
        if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&lin->state), bytes);
        if (e == cudaSuccess && d->grads) e = cudaMalloc(reinterpret_cast<void**>(&lin->dstate), bytes);
        if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&lin->d_err), 2 * sizeof(int));
        if (e == cudaSuccess) e = cudaMemset(lin->state, 0, bytes);
        if (e == cudaSuccess && d->grads) e = cudaMemset(lin->dstate, 0, bytes);
        if (e == cudaSuccess) e = cudaMemset(lin->d_err, 0, 2 * sizeof(int));
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
        if (e != cudaSuccess) {
            cudaGetLastError();
            pkv_lin_destroy(lin);
            return cuda_fail(e, "pkv_lin_create: states");
        }
        *out = lin;
        return PKV_OK;
    });
}

void pkv_lin_destroy(pkv_lin* lin) {
    if (!lin) return;
    if (lin->desc.residency != PKV_RES_META) {
        cudaFree(lin->state); cudaFree(lin->dstate); cudaFree(lin->d_err); cudaFree(lin->scratch);
        for (float* p : lin->retired) cudaFree(p);
    }
    delete lin;
}

pkv_status pkv_lin_arrays(const pkv_lin* lin, float** state, float** dstate) {
    if (!lin) return fail(PKV_ERR_INVALID, "pkv_lin_arrays: lin is NULL");
    if (state) *state = lin->state;
    if (dstate) *dstate = lin->dstate;
    return PKV_OK;
}

pkv_status pkv_lin_check(pkv_lin* lin) {
    return guarded("pkv_lin_check", [&]() -> pkv_status {
        if (!lin) return fail(PKV_ERR_INVALID, "pkv_lin_check: lin is NULL");
        if (lin->desc.residency == PKV_RES_META) return PKV_OK;
        const pkv_status waits = take_device_error(lin->d_err + 1, "pkv_lin_check");
        if (waits != PKV_OK) return waits;
        return take_device_error(lin->d_err, "pkv_lin_check");
    });
}

pkv_status pkv_lin_attn_fwd(pkv_lin* lin, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, void* o, int64_t o_stride, int64_t n, const float* log_decay,
                            const pkv_lin_batch* batch, void* stream) {
    static const char* who = "pkv_lin_attn_fwd";
    return guarded(who, [&]() -> pkv_status {
        LinArgs a{};
        pkv_status st = begin(lin, n, log_decay, &a, who);
        if (st == PKV_OK) st = batch_args(batch, &a, who);
        if (st != PKV_OK) return st;
        if (n > 0) {
            if ((st = operand(lin, q, a.Hq, q_stride, &a.q, who, "q")) != PKV_OK) return st;
            if ((st = operand(lin, k, a.Hkv, k_stride, &a.k, who, "k")) != PKV_OK) return st;
            if ((st = operand(lin, v, a.Hkv, v_stride, &a.v, who, "v")) != PKV_OK) return st;
            if ((st = operand(lin, o, a.Hq, o_stride, &a.o, who, "o")) != PKV_OK) return st;
        }
        if ((st = on_device(lin, who)) != PKV_OK || a.n_seq == 0) return st;
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if ((st = chunk_states(lin, &a, false, cs, who)) != PKV_OK) return st;
        std::string why;
        return launched(on_tensor_cores(lin) ? launch_lin_fwd_tc(a, cs, &why) : launch_lin_fwd_simt(a, cs), why, who);
    });
}

pkv_status pkv_lin_attn_bwd(pkv_lin* lin, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const void* dout, int64_t dout_stride, void* dq, int64_t dq_stride, void* dk,
                            int64_t dk_stride, void* dv, int64_t dv_stride, int64_t n, const float* log_decay,
                            const pkv_lin_batch* batch, void* stream) {
    static const char* who = "pkv_lin_attn_bwd";
    return guarded(who, [&]() -> pkv_status {
        LinArgs a{};
        pkv_status st = begin(lin, n, log_decay, &a, who);
        if (st == PKV_OK) st = batch_args(batch, &a, who);
        if (st != PKV_OK) return st;
        if (!lin->desc.grads) return fail(PKV_ERR_INVALID, "pkv_lin_attn_bwd: the store was created without gradients");
        if (n > 0) {
            if ((st = operand(lin, q, a.Hq, q_stride, &a.q, who, "q")) != PKV_OK) return st;
            if ((st = operand(lin, k, a.Hkv, k_stride, &a.k, who, "k")) != PKV_OK) return st;
            if ((st = operand(lin, v, a.Hkv, v_stride, &a.v, who, "v")) != PKV_OK) return st;
            if ((st = operand(lin, dout, a.Hq, dout_stride, &a.dout, who, "dout")) != PKV_OK) return st;
            if ((st = operand(lin, dq, a.Hq, dq_stride, &a.dq, who, "dq")) != PKV_OK) return st;
            if ((st = operand(lin, dk, a.Hkv, dk_stride, &a.dk, who, "dk")) != PKV_OK) return st;
            if ((st = operand(lin, dv, a.Hkv, dv_stride, &a.dv, who, "dv")) != PKV_OK) return st;
        }
        if ((st = on_device(lin, who)) != PKV_OK || a.n_seq == 0) return st;
        cudaStream_t cs = static_cast<cudaStream_t>(stream);
        if ((st = chunk_states(lin, &a, true, cs, who)) != PKV_OK) return st;
        std::string why;
        return launched(on_tensor_cores(lin) ? launch_lin_bwd_tc(a, cs, &why) : launch_lin_bwd_simt(a, cs), why, who);
    });
}

pkv_status pkv_lin_attn_step(pkv_lin* lin, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, void* o, int64_t o_stride, int64_t n, const float* log_decay,
                             const int32_t* slots, void* stream) {
    static const char* who = "pkv_lin_attn_step";
    return guarded(who, [&]() -> pkv_status {
        LinArgs a{};
        pkv_status st = begin(lin, n, log_decay, &a, who);
        if (st != PKV_OK) return st;
        if (n > 0) {
            if (!slots || misaligned(slots, 4)) return fail(PKV_ERR_INVALID, "pkv_lin_attn_step: slots is NULL or misaligned");
            if ((st = operand(lin, q, a.Hq, q_stride, &a.q, who, "q")) != PKV_OK) return st;
            if ((st = operand(lin, k, a.Hkv, k_stride, &a.k, who, "k")) != PKV_OK) return st;
            if ((st = operand(lin, v, a.Hkv, v_stride, &a.v, who, "v")) != PKV_OK) return st;
            if ((st = operand(lin, o, a.Hq, o_stride, &a.o, who, "o")) != PKV_OK) return st;
            if (n * a.Hkv > kMaxGrid / 4) return fail(PKV_ERR_UNSUPPORTED, "pkv_lin_attn_step: too many rows");
        }
        if ((st = on_device(lin, who)) != PKV_OK || n == 0) return st;
        a.slots = slots;
        const cudaError_t e = launch_lin_step(a, static_cast<cudaStream_t>(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "pkv_lin_attn_step: launch");
    });
}

}  // extern "C"
