"""The attention block with rotation and modified scores, trained chunk by chunk
through the library, against the same block as one float64 autograd graph over
the whole sequence: the rotated append, attention, its backward and the rotated
gradients together, with activation recomputation.

Tolerances (relative Frobenius) as for the plain block: 1e-4 in fp32, 2e-2 in
bf16 (bf16 projections whose inputs are rounded once, by 2^-8 relative at most, several
times in a row)."""
import math

import numpy as np
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build
from paged_kv_chunk_chunked_gb300 import synth
from paged_kv_chunk_chunked_gb300.layer import ChunkRecurrentBlock
from paged_kv_chunk_chunked_gb300.sweep import to_device, to_numpy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _whole_sequence(w, x, W, dy, inv_freq, interleaved, softcap, slopes, starts):
    """y, dx and the weight gradients in float64 on the CPU, by autograd."""
    t = lambda a: torch.tensor(a, dtype=torch.float64, requires_grad=True)  # noqa: E731
    x, W = t(x), {n: t(a) for n, a in W.items()}
    N, g = w.N, w.Hq // w.Hkv
    i = torch.arange(N)
    first = torch.zeros(N, dtype=torch.int64)
    for s in starts or [0]:
        first[s:] = s
    q, k, v = ((x @ W[n]).view(N, h, w.d) for n, h in (("wq", w.Hq), ("wk", w.Hkv), ("wv", w.Hkv)))
    if inv_freq is not None:
        ang = (i - first).double()[:, None, None] * inv_freq.double()
        c, s = ang.cos(), ang.sin()
        half = len(inv_freq)

        def turn(z):
            r, rest = z[..., :2 * half], z[..., 2 * half:]
            a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
            y = (a * c - b * s, b * c + a * s)
            y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
            return torch.cat([y, rest], -1)
        q, k = turn(q), turn(k)
    sc = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1)) / math.sqrt(w.d)
    if softcap:
        sc = softcap * torch.tanh(sc / softcap)
    if slopes is not None:
        sc = sc - slopes.double()[:, None, None] * (i[:, None] - i).abs()
    sc = sc.masked_fill((i[None] > i[:, None]) | (i[None] < first[:, None]), -math.inf)
    a = torch.einsum("hij,jhd->ihd", sc.softmax(-1), v.repeat_interleave(g, 1)).reshape(N, -1)
    y = x + a @ W["wo"]
    y.backward(torch.tensor(dy, dtype=torch.float64))
    return y.detach().numpy(), {"x": x.grad.numpy(), **{n: p.grad.numpy() for n, p in W.items()}}


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("key,kw,hidden,tol,rotary,inter,softcap,bias,starts", [
    ("tiny_dense_f32", {}, 64, 1e-4, 64, False, 2.0, True, [0, 100, 101, 190]),
    ("tiny_dense_f32", dict(N=200), 48, 1e-4, 32, True, 0.0, False, None),
    ("tiny_dense_f32", dict(N=150, Hq=4, Hkv=2), 48, 1e-4, 0, False, 0.0, True, [0, 64, 70]),
    ("qwen7b_dense_32k", dict(N=1152, C=256, Hq=4, Hkv=2), 256, 2e-2, 128, False, 1.0, False, [0, 300, 900]),
    ("qwen7b_dense_128k_perm", dict(N=1000, C=384, Hq=7, Hkv=1, extra_pages=3), 192, 2e-2, 64, True, 0.0, True, None),
    ("qwen7b_dense_32k", dict(N=640, C=256, Hq=8, Hkv=4, d=64), 128, 2e-2, 64, False, 0.0, False, [0, 513]),
])
def test_block_matches_whole_sequence(key, kw, hidden, tol, rotary, inter, softcap, bias, starts):
    w = synth.workload(key, **kw)
    n = w.n_chunks
    xs = [synth.block_x(w, c, hidden) for c in range(n)]
    dys = [synth.block_dy(w, c, hidden) for c in range(n)]
    inv_freq = torch.tensor([1e4 ** (-2.0 * i / rotary) for i in range(rotary // 2)]) if rotary else None
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / w.Hq) for h in range(w.Hq)]) if bias else None
    y_ref, g_ref = _whole_sequence(w, np.concatenate(xs), synth.block_weights(w, hidden), np.concatenate(dys), inv_freq, inter,
                                   softcap, slopes, starts)
    blk = ChunkRecurrentBlock(w, hidden, inv_freq=inv_freq, interleaved=inter, softcap=softcap, slopes=slopes, doc_starts=starts)
    try:
        xd, dyd = ([to_device(x, w.dtype) for x in a] for a in (xs, dys))
        for _ in range(2):                                   # a second step repeats the first
            ys = blk.forward(xd)
            dxs, grads = blk.backward(xd, dyd)
            torch.cuda.synchronize()
            B.pkv_check(blk.pool)
            err = {"y": _rel(np.concatenate([to_numpy(y) for y in ys]), y_ref),
                   "x": _rel(np.concatenate([to_numpy(d) for d in dxs]), g_ref["x"])}
            for name in ("wq", "wk", "wv", "wo"):
                err[name] = _rel(to_numpy(grads[name]), g_ref[name])
            assert max(err.values()) <= tol, err
    finally:
        blk.close()


def test_changed_weights_are_used_at_once():
    """Weights updated in place and replaced between two steps: the second step's
    outputs and gradients are those of the new weights throughout."""
    w, hidden = synth.workload("tiny_dense_f32", N=200), 48
    xs = [synth.block_x(w, c, hidden) for c in range(w.n_chunks)]
    dys = [synth.block_dy(w, c, hidden) for c in range(w.n_chunks)]
    inv_freq = torch.tensor([1e4 ** (-2.0 * i / w.d) for i in range(w.d // 2)])
    blk = ChunkRecurrentBlock(w, hidden, inv_freq=inv_freq, softcap=2.0)
    try:
        xd, dyd = ([to_device(x, w.dtype) for x in a] for a in (xs, dys))
        blk.forward(xd)
        blk.backward(xd, dyd)
        g = torch.Generator().manual_seed(7)
        for name in ("wq", "wk", "wo"):                      # as an optimiser's step
            t = blk.weights[name]
            t.add_((torch.randn(t.shape, generator=g) * t.std().item()).cuda())
        blk.weights["wv"] = blk.weights["wv"] * -0.5         # as a loaded checkpoint
        y_ref, g_ref = _whole_sequence(w, np.concatenate(xs), {n: to_numpy(t) for n, t in blk.weights.items()},
                                       np.concatenate(dys), inv_freq, False, 2.0, None, None)
        ys = blk.forward(xd)
        dxs, grads = blk.backward(xd, dyd)
        torch.cuda.synchronize()
        B.pkv_check(blk.pool)
        err = {"y": _rel(np.concatenate([to_numpy(y) for y in ys]), y_ref),
               "x": _rel(np.concatenate([to_numpy(d) for d in dxs]), g_ref["x"])}
        for name in ("wq", "wk", "wv", "wo"):
            err[name] = _rel(to_numpy(grads[name]), g_ref[name])
        assert max(err.values()) <= 1e-4, err
    finally:
        blk.close()


def test_generation_after_a_prefilled_chunk():
    """A chunk appended and attended at once, then tokens one at a time: each step's
    output is the whole sequence's row. Bounds as between two bf16 runs of the same
    keys: P and O rounded to bf16 in both (2 * 2^-8 of sum p |v|, and 2^-8 |o| twice)."""
    Hq, Hkv, d, P, n0, steps = 8, 2, 64, 128, 300, 5
    N = n0 + steps
    g = torch.Generator().manual_seed(3)
    x = torch.randn(N, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    inv = torch.tensor([1e4 ** (-2.0 * i / d) for i in range(d // 2)], device="cuda")
    out = []
    for cuts in ([0, N], [0, n0] + list(range(n0 + 1, N + 1))):
        pool = B.pkv_pool_create(P, Hkv, Hq, d, B.PKV_BF16, -(-N // P))
        try:
            seq = B.pkv_seq_create(pool)
            st = torch.cuda.current_stream()
            o, lse = torch.empty(N, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(Hq, N, device="cuda")
            for a, b in zip(cuts, cuts[1:]):
                qr, part = torch.empty(b - a, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(Hq, b - a, device="cuda")
                B.pkv_append_rope(seq, q[a:b], qr, k[a:b], v[a:b], b - a, B.rope(inv, pos0=a), st)
                B.pkv_chunk_attn_mod_fwd(seq, qr, a, b - a, o[a:b], part, B.score_mod(30.0), None, st)
                lse[:, a:b] = part
            B.pkv_check(pool)
            out.append((o.double(), lse.double()))
        finally:
            B.pkv_pool_destroy(pool)
    vmax = v.double().abs().max().item()
    assert (out[0][0] - out[1][0]).abs().max().item() <= 6 * 2.0 ** -8 * vmax
    assert (out[0][1] - out[1][1]).abs().max().item() <= 1e-4


def test_bad_documents_are_refused():
    w = synth.workload("tiny_dense_f32")
    for starts in ([], [1, 5], [0, 5, 5], [0, 256]):
        with pytest.raises(ValueError):
            ChunkRecurrentBlock(w, 32, doc_starts=starts)


@pytest.mark.parametrize("cap", [-1.0, float("nan")])
def test_a_bad_cap_is_refused(cap):
    """Not run as the plain attention."""
    w = synth.workload("tiny_dense_f32")
    blk = ChunkRecurrentBlock(w, 32, softcap=cap)
    try:
        xs = [torch.zeros(w.C, 32, device="cuda")]
        with pytest.raises(B.PkvError, match="softcap"):
            blk.forward(xs)
    finally:
        blk.close()
