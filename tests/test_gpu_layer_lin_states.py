"""The linear block's states: what belongs to whom between a forward, single tokens and a backward."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import synth
from paged_kv_chunk_chunked_gb300.layer import LinearRecurrentBlock
from paged_kv_chunk_chunked_gb300.sweep import to_device
from test_gpu_lin import Memory, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("key,kw,hidden,starts", [
    ("tiny_dense_f32", dict(N=250), 48, None),
    ("tiny_dense_f32", dict(N=200, Hq=4, Hkv=2), 40, [0, 64, 70, 150]),
    ("qwen7b_dense_32k", dict(N=640, C=256, Hq=4, Hkv=2, d=64), 128, None),
])
def test_a_backward_leaves_the_states(key, kw, hidden, starts):
    """Tokens generated between a forward and its backward: the backward changes no state (the
    generation goes on from where it was) and its gradients are those without the tokens."""
    w = synth.workload(key, **kw)
    blk = LinearRecurrentBlock(w, hidden, torch.linspace(-0.2, -0.01, w.Hkv), doc_starts=starts)
    try:
        state = torch.as_tensor(Memory(B.pkv_lin_arrays(blk.lin)["state"], (w.n_chunks + 1, w.Hkv, w.d, w.d)), device="cuda")
        xs, dys = ([to_device(f(w, c, hidden), w.dtype) for c in range(w.n_chunks)] for f in (synth.block_x, synth.block_dy))
        blk.forward(xs)
        want = blk.backward(xs, dys)
        blk.forward(xs)
        slot = torch.tensor([w.n_chunks], dtype=torch.int32, device="cuda")
        end = state[-1].clone()
        for t in range(3):
            blk.step(xs[0][t:t + 1], slot)
        before = state.clone()
        assert not torch.equal(before[-1], end)
        got = blk.backward(xs, dys)
        B.pkv_lin_check(blk.lin)
        assert torch.equal(state, before)
        assert all(torch.equal(a, b) for a, b in zip(got[0], want[0]))
        assert all(torch.equal(got[1][n], want[1][n]) for n in want[1])
    finally:
        blk.close()
