"""Chunk-recurrent training of one attention block on the paged KV cache, and of one
with linear attention, whose memory is a state instead.

The block is y = x + A wo, A = causal GQA attention(x wq, x wk, x wv), with
random weights (no data or trained model is involved). "Out of the Memory
Barrier" trains a layer chunk by chunk and recomputes activations in the
backward pass, so activation memory does not grow with the context; the KV
cache and its gradients live in pages and grow instead (gist.science/de §2.A
and §2.B; sciencestack.ai Fig. 1 and Fig. 3 captions). Here:

* forward, chunks in order: project the chunk, append its K/V to the paged
  cache (``pkv_append``), attend (``pkv_chunk_attn_fwd``), output projection
  and residual. Nothing per chunk is kept.
* backward, chunks in reverse: recompute the chunk's Q and its attention
  output and LSE (``pkv_chunk_attn_fwd`` again, over the full cache: the
  kernel sees keys up to each query only), dA = dy wo^T,
  ``pkv_chunk_attn_bwd`` (dQ written; dK/dV added into the paged gradient
  pool), then the chunk's own dK/dV rows, final because every later chunk's
  backward has run, are read out (``pkv_gather_rows``) and go back through
  the K/V projections.

With a rotation (``inv_freq``) the three projections are one matmul whose
Q and K slices are rotated on their way into the cache (``pkv_append_rope``),
and the gradients come back rotated the other way and laid out for it
(``pkv_rope_grad``). With a score cap, a distance bias or packed documents
(``softcap``, ``slopes``, ``doc_starts``) attention runs with modified scores
(``pkv_chunk_attn_mod_fwd`` / ``_bwd``); positions count from 0 in each document.

With ``norm_eps`` the projections read a layer norm of x (``pkv_layer_norm_fwd`` /
``_bwd``, its weight's gradient added chunk by chunk); without, as in the benchmarks,
x itself: the block exercises the path's KV-side memory and compute, not a particular
model. The projections are plain torch matmuls (cuBLAS); every attention step runs in
the library's kernels.

``LinearRecurrentBlock`` is the block of a layer without pages: y = x + norm(A) wo
with A linear attention of a layer norm of x and a norm of its own for each head of
A. Chunk c starts from the state in slot c of the block's store and leaves slot
c + 1, so the backward sweep finds every chunk's first state again and hands the
states' gradients back through the same slots.
"""
from __future__ import annotations

import torch

from . import binding as B
from . import synth
from .sweep import to_device


def _dtype_of(w: synth.Workload):
    return (torch.bfloat16, B.PKV_BF16) if w.dtype == "bf16" else (torch.float32, B.PKV_F32)


def _first_tokens(w: synth.Workload, doc_starts):
    """Per token, its document's first token (int64, host)."""
    starts = torch.as_tensor(doc_starts, dtype=torch.int64)
    if starts.numel() == 0 or starts[0] != 0 or (starts.diff() <= 0).any() or starts[-1] >= w.N:
        raise ValueError("doc_starts must ascend from 0 and stay below the sequence's length")
    return starts[torch.searchsorted(starts, torch.arange(w.N), right=True) - 1]


class _Norm:
    """Layer norm of groups of columns by the block's weights `names` (weight, bias), as
    they are at each call."""

    def __init__(self, block, names, width: int, groups: int, eps: float):
        self.block, self.names, self.width, self.groups, self.eps = block, names, width, groups, float(eps)

    def _desc(self):
        weight, bias = (self.block.weights[n] for n in self.names)
        return B.norm(self.width, self.groups, self.eps, weight, bias, _dtype_of(self.block.w)[1])

    def forward(self, x, stream):
        """(y, mean, rstd) of rows x."""
        n = len(x)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        mean, rstd = (torch.empty((n, self.groups), dtype=torch.float32, device=x.device) for _ in range(2))
        B.pkv_layer_norm_fwd(x, y, mean, rstd, n, self._desc(), stream)
        return y, mean, rstd

    def backward(self, dy, x, mean, rstd, grads, stream):
        """dx; adds the weight's and bias's gradients to `grads`."""
        n, desc = len(x), self._desc()
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        scratch = torch.empty(max(1, B.pkv_layer_norm_scratch(desc, n)), dtype=torch.float32, device=x.device)
        dw, db = (grads[name] for name in self.names)
        B.pkv_layer_norm_bwd(dy, x, mean, rstd, dx, dw, db, n, desc, scratch, accumulate=True, stream=stream)
        return dx


class ChunkRecurrentBlock:
    """One attention block of workload ``w`` (heads, page size, chunk length,
    dtype) with hidden size ``hidden`` and the seeded weights of
    ``synth.block_weights``; a paged pool holding one sequence of w.N tokens."""

    def __init__(self, w: synth.Workload, hidden: int, flags: int = 0, *, inv_freq=None,
                 interleaved: bool = False, softcap: float = 0.0, slopes=None, doc_starts=None,
                 norm_eps=None):
        """inv_freq: float32 [rotary_dim / 2] or None (no rotation). softcap, slopes
        (float32 [Hq]), doc_starts (ascending first tokens of the packed documents,
        from 0 on): the scores' modification; none of them is the plain attention.
        norm_eps: of the layer norm before the projections, with the weights norm_w
        (ones at first) and norm_b (zeros); None: no norm."""
        self.w, self.hidden = w, hidden
        self.inv_freq = None if inv_freq is None else inv_freq.to("cuda", torch.float32).contiguous()
        self.interleaved, self.softcap = interleaved, float(softcap)
        self.slopes = None if slopes is None else slopes.to("cuda", torch.float32).contiguous()
        self.first = None                        # per token: its document's first token
        if doc_starts is not None:
            self.first = _first_tokens(w, doc_starts).cuda()
        self.modified = self.softcap != 0 or slopes is not None or doc_starts is not None
        self.dt, pdt = _dtype_of(w)
        self.weights = {n: to_device(a, w.dtype) for n, a in synth.block_weights(w, hidden).items()}
        self.norm = None
        if norm_eps is not None:
            self.weights.update(norm_w=torch.ones(hidden, dtype=self.dt, device="cuda"),
                                norm_b=torch.zeros(hidden, dtype=self.dt, device="cuda"))
            self.norm = _Norm(self, ("norm_w", "norm_b"), hidden, 1, norm_eps)
        torch.cuda.synchronize()
        free0 = torch.cuda.mem_get_info()[0]
        self.pool = B.pkv_pool_create(w.P, w.Hkv, w.Hq, w.d, pdt, w.n_phys, flags=flags)
        torch.cuda.synchronize()
        self.pool_device_bytes = free0 - torch.cuda.mem_get_info()[0]   # K, V, dK, dV pages, reps
        self.seq = B.pkv_seq_create(self.pool)
        C = w.C
        self.o = torch.empty((C, w.Hq, w.d), dtype=self.dt, device="cuda")
        self._lse = torch.empty(w.Hq * C, dtype=torch.float32, device="cuda")
        self.dq = torch.empty((C, w.Hq, w.d), dtype=self.dt, device="cuda")
        self.dk = torch.empty((C, w.Hkv, w.d), dtype=torch.float32, device="cuda")
        self.dv = torch.empty_like(self.dk)
        if self.inv_freq is not None:
            heads = w.Hq + 2 * w.Hkv
            self.q = torch.empty((C, w.Hq, w.d), dtype=self.dt, device="cuda")
            self.dqkv = torch.empty((C, heads, w.d), dtype=self.dt, device="cuda")

    def _rope(self, s: int, e: int):
        if self.first is None:
            return B.rope(self.inv_freq, pos0=s, interleaved=self.interleaved)
        pos = torch.arange(s, e, device="cuda") - self.first[s:e]
        return B.rope(self.inv_freq, positions=pos, interleaved=self.interleaved)

    def _wqkv(self):
        """wq, wk and wv side by side, as they are now: formed once per forward or
        backward of the sequence, never kept, since training changes ``weights``."""
        return torch.cat([self.weights[n] for n in ("wq", "wk", "wv")], dim=1)

    def _qkv(self, x, wqkv):
        """Q, K and V [n, heads, d] as slices of one projection's output."""
        w = self.w
        return (x @ wqkv).view(len(x), -1, w.d).split([w.Hq, w.Hkv, w.Hkv], dim=1)

    def _attend(self, q, s: int, e: int, stream):
        n = e - s
        o, lse = self.o[:n], self._lse_of(n)
        if self.modified:
            B.pkv_chunk_attn_mod_fwd(self.seq, q, s, n, o, lse, self._mod(s, e), None, stream)
        else:
            B.pkv_chunk_attn_fwd(self.seq, q, s, n, o, lse, None, stream)
        return o, lse

    def _mod(self, s: int, e: int):
        return B.score_mod(self.softcap, self.slopes, None if self.first is None else self.first[s:e])

    def _lse_of(self, n: int) -> torch.Tensor:
        """[Hq, n] float32, contiguous (a partial last chunk has n < C)."""
        return self._lse[: self.w.Hq * n].view(self.w.Hq, n)

    def _reset(self):
        B.pkv_seq_reset(self.seq)
        if self.w.table == "perm":
            B.pkv_set_block_table(self.seq, synth.block_table(self.w))

    def forward(self, xs: list) -> list:
        """Chunks in order, on the current stream; returns every chunk's output y."""
        w, W = self.w, self.weights
        stream = torch.cuda.current_stream()
        self._reset()
        wqkv = self._wqkv() if self.inv_freq is not None else None
        ys = []
        for c, x in enumerate(xs):
            s, e = w.chunk_range(c)
            n = e - s
            y, x = x, x if self.norm is None else self.norm.forward(x, stream)[0]
            if self.inv_freq is not None:
                xq, k, v = self._qkv(x, wqkv)
                q = self.q[:n]
                B.pkv_append_rope(self.seq, xq, q, k, v, n, self._rope(s, e), stream)
            else:
                q = (x @ W["wq"]).view(n, w.Hq, w.d)
                k = (x @ W["wk"]).view(n, w.Hkv, w.d)
                v = (x @ W["wv"]).view(n, w.Hkv, w.d)
                B.pkv_append(self.seq, k, v, n, stream)
            o, _ = self._attend(q, s, e, stream)
            ys.append(y + o.view(n, -1) @ W["wo"])
        return ys

    def backward(self, xs: list, dys: list):
        """Chunks in reverse, on the current stream, after ``forward`` of the same
        inputs. Returns every chunk's input gradient and the weight gradients
        (float32)."""
        w, W = self.w, self.weights
        stream = torch.cuda.current_stream()
        g = {n: torch.zeros(t.shape, dtype=torch.float32, device="cuda") for n, t in W.items()}
        dxs = [None] * len(xs)
        wqkv = self._wqkv() if self.inv_freq is not None else None
        for c in reversed(range(len(xs))):
            s, e = w.chunk_range(c)
            n = e - s
            x, dy = xs[c], dys[c]
            if self.norm is not None:
                x, *stats = self.norm.forward(x, stream)              # recomputed
            q = (x @ W["wq"]).view(n, w.Hq, w.d)                      # recomputed
            if self.inv_freq is not None:
                B.pkv_rope_rows(self.pool, q, q, n, w.Hq, self._rope(s, e), stream=stream)
            o, lse = self._attend(q, s, e, stream)                    # recomputed
            dq = self.dq[:n]
            a = o.view(n, -1)
            da = (dy @ W["wo"].t()).view(n, w.Hq, w.d)
            g["wo"] += (a.t() @ dy).float()
            if self.modified:
                B.pkv_chunk_attn_mod_bwd(self.seq, q, o, da, lse, s, n, dq, self._mod(s, e), None, stream)
            else:
                B.pkv_chunk_attn_bwd(self.seq, q, o, da, lse, s, n, dq, None, stream)
            xt = x.t()
            if self.inv_freq is not None:
                # rows s..e-1 are final, as below
                parts = self.dqkv[:n].split([w.Hq, w.Hkv, w.Hkv], dim=1)
                B.pkv_rope_grad(self.seq, s, n, self._rope(s, e), dq, *parts, stream=stream)
                d = self.dqkv[:n].view(n, -1)
                dxs[c] = self._dx(dy, d @ wqkv.t(), xs[c], stats if self.norm else None, g, stream)
                gw = (xt @ d).float().split([W[name].shape[1] for name in ("wq", "wk", "wv")], dim=1)
                for name, part in zip(("wq", "wk", "wv"), gw):
                    g[name] += part
                continue
            # rows s..e-1 of dK/dV are final: no earlier chunk's queries see them
            B.pkv_gather_rows(self.seq, s, n, None, None, self.dk[:n], self.dv[:n], stream)
            dqf = dq.view(n, -1)
            dkf = self.dk[:n].view(n, -1).to(self.dt)
            dvf = self.dv[:n].view(n, -1).to(self.dt)
            if self.norm is None:
                dxs[c] = dy + dqf @ W["wq"].t() + dkf @ W["wk"].t() + dvf @ W["wv"].t()
            else:
                dxs[c] = self._dx(dy, dqf @ W["wq"].t() + dkf @ W["wk"].t() + dvf @ W["wv"].t(), xs[c], stats, g, stream)
            g["wq"] += (xt @ dqf).float()
            g["wk"] += (xt @ dkf).float()
            g["wv"] += (xt @ dvf).float()
        return dxs, g

    def _dx(self, dy, dh, x, stats, grads, stream):
        """The input's gradient: through the residual and from the projections' input's dh."""
        return dy + (dh if self.norm is None else self.norm.backward(dh, x, *stats, grads, stream))

    def close(self):
        if self.pool:
            B.pkv_pool_destroy(self.pool)
            self.pool = 0


class LinearRecurrentBlock:
    """One block with linear attention of workload ``w`` (heads, chunk length, dtype)
    with hidden size ``hidden`` and the seeded projections of ``synth.block_weights``:
    y = x + norm(A) wo, A the linear attention of norm(x) (wq, wk, wv), normalised for
    each head. A store holds one state more than the sequence has chunks."""

    def __init__(self, w: synth.Workload, hidden: int, log_decay, eps: float = 1e-5, doc_starts=None, flags: int = 0):
        """log_decay: float32 [Hkv], the natural logs of the heads' decays, or None (no
        decay). doc_starts: ascending first tokens of packed documents, from 0 on; no
        state is carried from one into the next."""
        self.w, self.hidden = w, hidden
        self.dt, kind = _dtype_of(w)
        self.log_decay = None if log_decay is None else log_decay.to("cuda", torch.float32).contiguous()
        self.first = None if doc_starts is None else _first_tokens(w, doc_starts)
        self.weights = {n: to_device(a, w.dtype) for n, a in synth.block_weights(w, hidden).items()}
        for name, cols in (("norm", hidden), ("head", w.Hq * w.d)):
            self.weights[name + "_w"] = torch.ones(cols, dtype=self.dt, device="cuda")
            self.weights[name + "_b"] = torch.zeros(cols, dtype=self.dt, device="cuda")
        self.norm = _Norm(self, ("norm_w", "norm_b"), hidden, 1, eps)
        self.head_norm = _Norm(self, ("head_w", "head_b"), w.d, w.Hq, eps)
        self.lin = B.pkv_lin_create(w.Hkv, w.Hq, w.d, kind, w.n_chunks + 1, grads=True, flags=flags)
        self._batches = {}

    def _batch(self, c: int):
        """Chunk c's sequences: pieces of documents. The first goes on from slot c if its
        document began before the chunk, the last leaves slot c + 1 if its goes on after it.
        Of the forward, of its recomputation (which leaves no state) and of the backward."""
        if c not in self._batches:
            s, e = self.w.chunk_range(c)
            first = self.first
            cuts = [s] if first is None else [s] + [t for t in range(s + 1, e) if first[t] == t]
            goes_on = (lambda t: 0 < t < self.w.N) if first is None else (lambda t: 0 < t < self.w.N and first[t] != t)
            m = len(cuts)
            slot_in, slot_out = [-1] * m, [-1] * m
            slot_in[0] = c if goes_on(s) else -1
            # (the last chunk's state is kept too: generation goes on from it)
            slot_out[-1] = c + 1 if goes_on(e) or e == self.w.N else -1
            back = list(slot_out)
            back[-1] = c + 1 if goes_on(e) else -1               # no gradient comes from behind the end
            dev = lambda a, t: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
            cu, at = dev([t - s for t in cuts] + [e - s], torch.int64), dev(slot_in, torch.int32)
            self._batches[c] = tuple(B.lin_batch(m, cu, at, None if out is None else dev(out, torch.int32))
                                     for out in (slot_out, None, back))
        return self._batches[c]

    def _check_rows(self, c: int, x):
        s, e = self.w.chunk_range(c)
        if len(x) != max(0, e - s):
            raise ValueError(f"chunk {c} has {max(0, e - s)} rows, got {len(x)}")

    def _qkv(self, h):
        w = self.w
        return [(h @ self.weights[name]).view(len(h), -1, w.d) for name in ("wq", "wk", "wv")]

    def forward(self, xs: list) -> list:
        """Chunks in order, on the current stream; returns every chunk's output y."""
        stream = torch.cuda.current_stream()
        ys = []
        for c, x in enumerate(xs):
            self._check_rows(c, x)
            h, _, _ = self.norm.forward(x, stream)
            q, k, v = self._qkv(h)
            a = torch.empty_like(q)
            B.pkv_lin_attn_fwd(self.lin, q, k, v, a, len(x), self.log_decay, self._batch(c)[0], stream)
            z, _, _ = self.head_norm.forward(a.view(len(x), -1), stream)
            ys.append(x + z @ self.weights["wo"])
        return ys

    def backward(self, xs: list, dys: list):
        """Chunks in reverse, on the current stream, after ``forward`` of the same inputs
        (activations are recomputed, from the states that it left; the backward writes none, so
        tokens may be generated in between). Returns every chunk's input gradient and the
        weight gradients (float32)."""
        if len(xs) != self.w.n_chunks or len(dys) != len(xs):
            raise ValueError(f"the backward goes over all {self.w.n_chunks} chunks, got {len(xs)} and {len(dys)}")
        W, stream = self.weights, torch.cuda.current_stream()
        g = {n: torch.zeros(t.shape, dtype=torch.float32, device="cuda") for n, t in W.items()}
        dxs = [None] * len(xs)
        for c in reversed(range(len(xs))):
            x, dy, n = xs[c], dys[c], len(xs[c])
            self._check_rows(c, x)
            _, again, back = self._batch(c)
            h, *stats = self.norm.forward(x, stream)
            q, k, v = self._qkv(h)
            a = torch.empty_like(q)
            B.pkv_lin_attn_fwd(self.lin, q, k, v, a, n, self.log_decay, again, stream)
            a = a.view(n, -1)
            z, *head_stats = self.head_norm.forward(a, stream)
            g["wo"] += (z.t() @ dy).float()
            da = self.head_norm.backward(dy @ W["wo"].t(), a, *head_stats, g, stream).view(q.shape)
            dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
            B.pkv_lin_attn_bwd(self.lin, q, k, v, da, dq, dk, dv, n, self.log_decay, back, stream)
            dh = 0
            for name, d in (("wq", dq), ("wk", dk), ("wv", dv)):
                d = d.view(n, -1)
                g[name] += (h.t() @ d).float()
                dh = dh + d @ W[name].t()
            dxs[c] = dy + self.norm.backward(dh, x, *stats, g, stream)
        return dxs, g

    def step(self, x, slots):
        """One token for each of a batch: x [n, hidden], slots int32 [n], the state each
        goes on from and advances (``n_chunks`` after ``forward``: the sequence's end)."""
        n, stream = len(x), torch.cuda.current_stream()
        h, _, _ = self.norm.forward(x, stream)
        q, k, v = self._qkv(h)
        a = torch.zeros_like(q)
        B.pkv_lin_attn_step(self.lin, q, k, v, a, n, self.log_decay, slots, stream)
        z, _, _ = self.head_norm.forward(a.view(n, -1), stream)
        return x + z @ self.weights["wo"]

    def close(self):
        if self.lin:
            torch.cuda.synchronize()
            B.pkv_lin_destroy(self.lin)
            self.lin = 0
