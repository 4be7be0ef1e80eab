"""Chunk-recurrent training of one attention block on the paged KV cache.

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

No normalisation: the block exercises the path's KV-side memory and compute, not
a particular model. The projections are plain torch matmuls (cuBLAS); every
attention step runs in the library's kernels.
"""
from __future__ import annotations

import torch

from . import binding as B
from . import synth
from .sweep import to_device


class ChunkRecurrentBlock:
    """One attention block of workload ``w`` (heads, page size, chunk length,
    dtype) with hidden size ``hidden`` and the seeded weights of
    ``synth.block_weights``; a paged pool holding one sequence of w.N tokens."""

    def __init__(self, w: synth.Workload, hidden: int, flags: int = 0, *, inv_freq=None,
                 interleaved: bool = False, softcap: float = 0.0, slopes=None, doc_starts=None):
        """inv_freq: float32 [rotary_dim / 2] or None (no rotation). softcap, slopes
        (float32 [Hq]), doc_starts (ascending first tokens of the packed documents,
        from 0 on): the scores' modification; none of them is the plain attention."""
        self.w, self.hidden = w, hidden
        self.inv_freq = None if inv_freq is None else inv_freq.to("cuda", torch.float32).contiguous()
        self.interleaved, self.softcap = interleaved, float(softcap)
        self.slopes = None if slopes is None else slopes.to("cuda", torch.float32).contiguous()
        self.first = None                        # per token: its document's first token
        if doc_starts is not None:
            starts = torch.as_tensor(doc_starts, dtype=torch.int64)
            if starts.numel() == 0 or starts[0] != 0 or (starts.diff() <= 0).any() or starts[-1] >= w.N:
                raise ValueError("doc_starts must ascend from 0 and stay below the sequence's length")
            self.first = starts[torch.searchsorted(starts, torch.arange(w.N), right=True) - 1].cuda()
        self.modified = self.softcap != 0 or slopes is not None or doc_starts is not None
        self.dt = torch.bfloat16 if w.dtype == "bf16" else torch.float32
        self.weights = {n: to_device(a, w.dtype) for n, a in synth.block_weights(w, hidden).items()}
        pdt = B.PKV_BF16 if w.dtype == "bf16" else B.PKV_F32
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
            ys.append(x + o.view(n, -1) @ W["wo"])
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
                dxs[c] = dy + d @ wqkv.t()
                gw = (xt @ d).float().split([W[name].shape[1] for name in ("wq", "wk", "wv")], dim=1)
                for name, part in zip(("wq", "wk", "wv"), gw):
                    g[name] += part
                continue
            # rows s..e-1 of dK/dV are final: no earlier chunk's queries see them
            B.pkv_gather_rows(self.seq, s, n, None, None, self.dk[:n], self.dv[:n], stream)
            dqf = dq.view(n, -1)
            dkf = self.dk[:n].view(n, -1).to(self.dt)
            dvf = self.dv[:n].view(n, -1).to(self.dt)
            dxs[c] = dy + dqf @ W["wq"].t() + dkf @ W["wk"].t() + dvf @ W["wv"].t()
            g["wq"] += (xt @ dqf).float()
            g["wk"] += (xt @ dkf).float()
            g["wv"] += (xt @ dvf).float()
        return dxs, g

    def close(self):
        if self.pool:
            B.pkv_pool_destroy(self.pool)
            self.pool = 0
