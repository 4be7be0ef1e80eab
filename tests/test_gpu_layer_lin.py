"""The blocks with linear attention and with layer norm, trained chunk by chunk through
the library, against the same blocks as one float64 autograd graph over the whole
sequence: norm, projections, attention and their backward passes together, with
activation recomputation and states carried from chunk to chunk.

Tolerances (relative Frobenius) as for the other blocks: 1e-4 in fp32; in bf16 2e-2
for what passes about ten roundings of 2^-9 rms each, most of them in projections."""
import math

import numpy as np
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build
from paged_kv_chunk_chunked_gb300 import synth
from paged_kv_chunk_chunked_gb300.layer import ChunkRecurrentBlock, LinearRecurrentBlock
from paged_kv_chunk_chunked_gb300.sweep import to_device, to_numpy

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _norm(x, w, b, eps):
    m = x.mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps) * w + b


def _whole(w, x, W, dy, weights, eps):
    """y, dx and the weight gradients in float64 on the CPU, by autograd; weights: [Hq, N, N], how
    query i sees key j (a function of the scores)."""
    t = lambda a: torch.tensor(a, dtype=torch.float64, requires_grad=True)  # noqa: E731
    x, W = t(x), {n: t(a) for n, a in W.items()}
    h = _norm(x, W["norm_w"], W["norm_b"], eps)
    N, g = w.N, w.Hq // w.Hkv
    q, k, v = ((h @ W[n]).view(N, -1, w.d) for n in ("wq", "wk", "wv"))
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1)) / math.sqrt(w.d)
    a = torch.einsum("hij,jhd->ihd", weights(s), v.repeat_interleave(g, 1))
    if "head_w" in W:
        a = _norm(a, W["head_w"].view(w.Hq, w.d), W["head_b"].view(w.Hq, w.d), eps)
    y = x + a.reshape(N, -1) @ W["wo"]
    y.backward(torch.tensor(dy, dtype=torch.float64))
    return y.detach().numpy(), {"x": x.grad.numpy(), **{n: p.grad.numpy() for n, p in W.items()}}


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def _run(blk, w, hidden, weights, tol, check):
    g = torch.Generator().manual_seed(11)
    for n, p in blk.weights.items():                         # norms that do something
        if n.endswith("_w") or n.endswith("_b"):
            p.add_((0.2 * torch.randn(p.shape, generator=g)).to(p.dtype).cuda())
    xs, dys = ([f(w, c, hidden) for c in range(w.n_chunks)] for f in (synth.block_x, synth.block_dy))
    xs = [x + 0.5 for x in xs] if w.dtype == "f32" else xs
    y_ref, g_ref = _whole(w, np.concatenate(xs), {n: to_numpy(p) for n, p in blk.weights.items()}, np.concatenate(dys), weights, 1e-5)
    xd, dyd = ([to_device(x, w.dtype) for x in a] for a in (xs, dys))
    for _ in range(2):                                       # a second step repeats the first
        ys = blk.forward(xd)
        dxs, grads = blk.backward(xd, dyd)
        torch.cuda.synchronize()
        check()
        err = {"y": _rel(np.concatenate([to_numpy(y) for y in ys]), y_ref),
               "x": _rel(np.concatenate([to_numpy(d) for d in dxs]), g_ref["x"])}
        for n in blk.weights:
            err[n] = _rel(to_numpy(grads[n]), g_ref[n])
        assert max(err.values()) <= tol, err
    return xd, ys


CASES = [
    ("tiny_dense_f32", dict(N=250), 48, 1e-4, None),
    ("tiny_dense_f32", dict(N=200, Hq=4, Hkv=2), 40, 1e-4, [0, 64, 70, 150]),
    ("qwen7b_dense_32k", dict(N=1000, C=384, Hq=7, Hkv=1), 192, 2e-2, [0, 300, 768]),
    ("qwen7b_dense_32k", dict(N=640, C=256, Hq=8, Hkv=4, d=64), 128, 2e-2, None),
]


@pytest.mark.parametrize("key,kw,hidden,tol,starts", CASES)
def test_linear_block_matches_whole_sequence(key, kw, hidden, tol, starts):
    w = synth.workload(key, **kw)
    log_decay = torch.linspace(-0.2, -0.01, w.Hkv)
    i = torch.arange(w.N)
    first = torch.zeros(w.N, dtype=torch.int64)
    for s in starts or [0]:
        first[s:] = s
    age = (i[:, None] - i).double()
    seen = (age >= 0) & (i[None] >= first[:, None])
    decay = torch.exp(log_decay.double().repeat_interleave(w.Hq // w.Hkv)[:, None, None] * age.clamp(min=0)) * seen
    blk = LinearRecurrentBlock(w, hidden, log_decay, doc_starts=starts)
    try:
        _run(blk, w, hidden, lambda s: s * decay, tol, lambda: B.pkv_lin_check(blk.lin))
    finally:
        blk.close()


@pytest.mark.parametrize("key,kw,hidden,tol,rotary", [
    ("tiny_dense_f32", dict(N=200), 48, 1e-4, 0),
    ("tiny_dense_f32", dict(N=200), 48, 1e-4, 64),
    ("qwen7b_dense_32k", dict(N=640, C=256, Hq=4, Hkv=2), 256, 2e-2, 0),
])
def test_normalised_attention_block(key, kw, hidden, tol, rotary):
    """The block on pages with a layer norm before its projections (a rotation of zero
    frequencies, so that its path through the rotated append runs too)."""
    w = synth.workload(key, **kw)
    i = torch.arange(w.N)
    inv = torch.zeros(rotary // 2) if rotary else None
    blk = ChunkRecurrentBlock(w, hidden, inv_freq=inv, norm_eps=1e-5)
    try:
        _run(blk, w, hidden, lambda s: s.masked_fill(i[None] > i[:, None], -math.inf).softmax(-1), tol, lambda: B.pkv_check(blk.pool))
    finally:
        blk.close()


def test_generation_goes_on_from_the_last_chunk():
    """Tokens one at a time after the chunks: the rows of a sequence that is longer by them."""
    w, hidden, steps = synth.workload("tiny_dense_f32", N=150), 48, 4
    longer = w.with_(N=150 + steps)
    log_decay = torch.tensor([-0.05])
    a, b = LinearRecurrentBlock(w, hidden, log_decay), LinearRecurrentBlock(longer, hidden, log_decay)
    try:
        xs = [to_device(synth.block_x(longer, c, hidden), "f32") for c in range(longer.n_chunks)]
        want = torch.cat(b.forward(xs))
        x = torch.cat(xs)
        a.forward([x[s:e] for s, e in (w.chunk_range(c) for c in range(w.n_chunks))])
        slots = torch.tensor([w.n_chunks, -1], dtype=torch.int32, device="cuda")
        for t in range(150, 150 + steps):
            y = a.step(x[t].expand(2, hidden).contiguous(), slots)
            # fp32 both, sums in another order: some 300 additions and a norm of the result.
            assert (y[0] - want[t]).abs().max().item() <= 1e-4 * want[t].abs().max().item()
        B.pkv_lin_check(a.lin)
    finally:
        a.close()
        b.close()


def test_bad_documents_are_refused():
    w = synth.workload("tiny_dense_f32")
    for starts in ([], [1, 5], [0, 5, 5], [0, 256]):
        with pytest.raises(ValueError):
            LinearRecurrentBlock(w, 32, None, doc_starts=starts)


def test_chunks_of_other_lengths_are_refused():
    w = synth.workload("tiny_dense_f32")
    blk = LinearRecurrentBlock(w, 32, None)
    try:
        xs = [torch.zeros(w.C, 32, device="cuda") for _ in range(w.n_chunks)]
        for bad in ([xs[0][:-1]], [xs[0], torch.cat(xs[:2])], xs + [xs[0]]):
            with pytest.raises(ValueError, match="rows"):
                blk.forward(bad)
        blk.forward(xs)
        with pytest.raises(ValueError, match="all"):
            blk.backward(xs[:-1], xs[:-1])
        blk.forward(xs[:2])                          # a beginning is allowed
    finally:
        blk.close()
