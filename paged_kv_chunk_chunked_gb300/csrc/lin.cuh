// Linear attention with a decay per head: what its kernels share.
//
//   S_t = l S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,   scale = 1 / sqrt(d)
//
// A sequence is cut into chunks of L rows. With S the state before a chunk of m
// rows, G the gradient of the state after it, and M_ij = l^(i-j) for j <= i, else 0:
//   O  = scale [((Q K^T) o M) V + diag(l^(i+1)) Q S]
//   dQ = scale [((dO V^T) o M) K + diag(l^(i+1)) dO S^T]
//   dV = scale ((Q K^T) o M)^T dO + diag(l^(m-1-j)) K G
//   dK = scale ((dO V^T) o M)^T Q + diag(l^(m-1-j)) V G^T
// (Q, dO of every query head of the group), and from chunk to chunk
//   S' = l^m S + sum_j l^(m-1-j) k_j v_j^T,   G' = l^m G + scale sum_i l^(i+1) q_i do_i^T.
// All exponents are >= 0, so nothing overflows for l <= 1, however long the chunk.
// O and dQ have one form, and dV and dK have one: "rows" and "columns" below.
#pragma once

#include "common.cuh"
#include "internal.h"

struct pkv_lin {
    pkv_lin_desc desc{};
    int device = 0;
    float* state = nullptr;          // [n_slots, Hkv, d, d]
    float* dstate = nullptr;         // the same, or null
    int* d_err = nullptr;            // two device error words: bad arguments, expired waits
    float* scratch = nullptr;        // chunk states, grown on demand; outgrown buffers stay until
    size_t scratch_floats = 0;       // the store is destroyed (a captured graph may use them)
    std::vector<float*> retired;
};

namespace pkv {

struct LinRows {
    void* p;                         // [n, heads, d], rows `stride` elements apart
    int64_t stride;
};

struct LinArgs {
    int Hq, Hkv, d, dtype;
    int64_t n, n_seq, n_slots;
    LinRows q, k, v, o, dout, dq, dk, dv;
    const float* log_decay;          // [Hkv] or null
    const int64_t* cu;               // [n_seq + 1] or null: one sequence of n rows
    const int32_t* slot_in;          // [n_seq] or null
    const int32_t* slot_out;         // [n_seq] or null
    const int32_t* slots;            // the step's, [n]
    float* state;
    float* dstate;
    float* part;                     // scratch [chunks, Hkv, d, d]: each chunk's sum, then the state before it
    float* gpart;                    // the same of the gradients: the gradient of the state after it
                                     // (tensor-core kernels: states and gradients as rows of d first and d second bf16 terms)
    int n_chunks;                    // lin_chunks
    bool one_term;                   // tensor-core kernels: PKV_FLAG_LIN_ONE_TERM
    int* err;                        // word of bad arguments
    int* wait_err;                   // word of the bounded waits: these give up once it is set
};

// Chunk numbers that n rows in n_seq sequences can take. Sequence b's chunks are
// numbered from cu[b] / L + b on: it has at most cu[b+1] / L - cu[b] / L + 1 of
// them, so no two sequences share a number and none needs a table.
inline int64_t lin_chunks(int64_t n, int64_t n_seq, int L) { return n / L + n_seq; }

// Whether rows lo .. hi - 1 are rows of the call (recorded if not).
__device__ __forceinline__ bool lin_good(const LinArgs& a, int64_t lo, int64_t hi) {
    if (lo >= 0 && lo <= hi && hi <= a.n) return true;
    report_error(a.err, kErrBadSeq);
    return false;
}

// The sequence's rows, checked.
__device__ __forceinline__ bool lin_range(const LinArgs& a, int64_t b, int64_t& lo, int64_t& hi) {
    lo = a.cu ? a.cu[b] : 0;
    hi = a.cu ? a.cu[b + 1] : a.n;
    return lin_good(a, lo, hi);
}

struct LinChunk {
    int row0;                        // first row (a call has less than 2^31)
    int rows;                        // 1 .. L
};

// The sequences' rows, of up to 32: kernels that look many chunks up load them once, into
// shared memory (registers are short where it is read).
struct LinCuts {
    int64_t lo[32], hi[32];
    // By one warp.
    __device__ __forceinline__ void load(const LinArgs& a) {
        const int64_t b = threadIdx.x % 32;
        const bool in = a.cu && b < a.n_seq;
        lo[b] = in ? a.cu[b] : 0;
        hi[b] = in ? a.cu[b + 1] : 0;
    }
};

// The rows of chunk number f; false: there is no such chunk. Called by whole warps.
// first: the sequences' rows (used if they are all there), or null.
template <int L> __device__ __forceinline__ bool lin_chunk(const LinArgs& a, const LinCuts* first, int f, LinChunk& c) {
    int64_t b = 0, lo = 0, hi = a.n;
    if (a.cu) {
        // The last sequence whose chunks start at or before f (numbers ascend with b): narrowed
        // down to 32 neighbours by 32 probes at a time, then found among them with its rows.
        const int lane = threadIdx.x % 32;
        int64_t len = a.n_seq;
        while (len > 32) {
            const int64_t step = (len + 31) / 32, x = b + lane * step;
            const int k = __popc(__ballot_sync(0xffffffffu, lane * step < len && a.cu[x] / L + x <= f));
            if (k == 0) return false;
            b += (k - 1) * step;
            len = min64(step, len - (k - 1) * step);
        }
        int64_t l = 0, r = 0;
        if (first && a.n_seq <= 32) {
            l = first->lo[lane];
            r = first->hi[lane];
        } else if (lane < len) {
            l = a.cu[b + lane];
            r = a.cu[b + lane + 1];
        }
        const int k = __popc(__ballot_sync(0xffffffffu, lane < len && l / L + b + lane <= f));
        if (k == 0) return false;
        lo = __shfl_sync(0xffffffffu, l, k - 1);
        hi = __shfl_sync(0xffffffffu, r, k - 1);
        b += k - 1;
    }
    if (!lin_good(a, lo, hi)) return false;
    const int64_t off = ((int64_t)f - (lo / L + b)) * L;
    if (off < 0 || off >= hi - lo) return false;
    c.row0 = (int)(lo + off);
    c.rows = (int)min64(L, hi - lo - off);
    return true;
}
template <int L> __device__ __forceinline__ bool lin_chunk(const LinArgs& a, int f, LinChunk& c) { return lin_chunk<L>(a, nullptr, f, c); }

__device__ __forceinline__ float lin_g2(const LinArgs& a, int kvh) {
    return a.log_decay ? a.log_decay[kvh] * kLog2e : 0.f;
}
// l^m, m >= 0, from log2 l (which may be -inf).
__device__ __forceinline__ float lin_pow(float g2, int m) { return m == 0 ? 1.f : exp2f(g2 * (float)m); }

// A sequence's slot, checked; -1 for none.
__device__ __forceinline__ int64_t lin_good_slot(const LinArgs& a, int32_t s) {
    if (s >= -1 && s < a.n_slots) return s;
    report_error(a.err, kErrBadSlot);
    return -1;
}
__device__ __forceinline__ int64_t lin_slot(const LinArgs& a, const int32_t* slots, int64_t b) {
    return slots ? lin_good_slot(a, slots[b]) : -1;
}

// By all threads of a CTA, for one sequence: records whether `mine`, which sequence b
// writes, is written for one before it or read for any other (`read` may be null). In calls
// of many sequences, where looking at all pairs would cost more than the states, it is left out.
constexpr int64_t kCheckedSeqs = 8192;
__device__ __forceinline__ void lin_check_alone(const LinArgs& a, const int32_t* written, const int32_t* read, int64_t b, int64_t mine,
                                                int64_t n) {
    if (mine < 0 || n > kCheckedSeqs) return;
    bool twice = false;
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
        if (j < b) twice |= written[j] == mine;
        if (read && j != b) twice |= read[j] == mine;
    }
    if (twice) report_error(a.err, kErrSlotTwice);
}

// CUDA-core kernels (chunks of kLinSimtChunk rows).
constexpr int kLinSimtChunk = 64;
cudaError_t launch_lin_fwd_simt(const LinArgs& a, cudaStream_t s);
cudaError_t launch_lin_bwd_simt(const LinArgs& a, cudaStream_t s);
// Tensor-core kernels (bf16, chunks of kLinTcChunk rows); *why: what failed other than a CUDA call.
constexpr int kLinTcChunk = 128;
cudaError_t launch_lin_fwd_tc(const LinArgs& a, cudaStream_t s, std::string* why);
cudaError_t launch_lin_bwd_tc(const LinArgs& a, cudaStream_t s, std::string* why);
cudaError_t launch_lin_step(const LinArgs& a, cudaStream_t s);

}  // namespace pkv
