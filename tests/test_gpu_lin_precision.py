"""bf16 linear attention on the tensor cores keeps its intermediate values to 16 bits: only the
outputs are rounded to bf16, unless the store's caller chose otherwise.

Bounds. mag is the sum of the terms' absolute values. F = (d + 224 + chunks) 2^-24 mag is the
float32 work's, as for the other linear attention tests. A chunk's weighted scores, the states that chunks start from and
their gradients are operands of bf16 products; each goes there as two bf16 terms, the first
off by half a step, 2^-8 of the value, and the second by 2^-8 of what is left: 2^-16 mag.
Storage rounds an output once: half a step. With PKV_FLAG_LIN_ONE_TERM the second term is left
out: 2^-8 mag."""
import numpy as np
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
import test_gpu_lin as base
from test_gpu_lin import Store, _close, _decays, _lib, _oracle, _rows  # noqa: F401

pytestmark = pytest.mark.gpu

TERMS = [(0, 2.0 ** -16), (B.PKV_FLAG_LIN_ONE_TERM, 2.0 ** -8)]
CASES = [
    # Hq, Hkv, d, cuts, decay, rows strided
    (4, 2, 128, [0, 1], "spread", False),
    (4, 2, 64, [0, 1], None, False),
    (7, 1, 128, [0, 300], "spread", True),
    (4, 4, 128, [0, 129, 129, 640], "zero", False),
    (4, 2, 64, [0, 127, 128, 128, 385], "spread", True),
    (6, 2, 128, [3, 67, 196, 196, 325, 330], "fast", False),
    (2, 2, 64, [0, 1000], None, True),
    (5, 1, 64, [7, 72], "own", False),
    (140, 70, 64, [2, 130, 150], "spread", False),       # more KV heads than the sums kernel's table of decays
]


def _inputs(Hq, Hkv, d, cuts, kind, strided):
    n, m = cuts[-1] + 5, len(cuts) - 1
    x = _rows(n, (Hq, Hkv, Hkv, Hq), d, torch.bfloat16, strided, n + d)
    log_decay = _decays(kind, Hkv)
    decay = np.ones(Hkv) if log_decay is None else np.exp(log_decay.double().numpy())
    r = np.random.default_rng(n)
    first, dlast = (r.standard_normal((m, Hkv, d, d)).astype(np.float32).astype(float) for _ in range(2))
    want, mag = _oracle(x, cuts, decay, first, dlast), _oracle(x, cuts, decay, first, dlast, np.abs)
    return n, m, x, None if log_decay is None else log_decay.cuda(), first, dlast, want, mag


def _fill(at, values):
    at.copy_(torch.tensor(values, dtype=torch.float32, device="cuda"))


@pytest.mark.parametrize("flags,off", TERMS)
@pytest.mark.parametrize("Hq,Hkv,d,cuts,kind,strided", CASES)
def test_forward(Hq, Hkv, d, cuts, kind, strided, flags, off):
    n, m, (q, k, v, _), g2, first, _, want, mag = _inputs(Hq, Hkv, d, cuts, kind, strided)
    with Store("bf16", Hq, Hkv, d, m, grads=False, flags=flags) as c:
        _fill(c.state, first)
        at = torch.arange(m, dtype=torch.int32, device="cuda")
        o = torch.full((n, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
        B.pkv_lin_attn_fwd(c.lin, q, k, v, o, n, g2, B.lin_batch(m, torch.tensor(cuts, device="cuda"), at, at),
                           torch.cuda.current_stream())
        B.pkv_lin_check(c.lin)
        s, F = slice(cuts[0], cuts[-1]), (d + 224 + n // 64) * 2.0 ** -24
        _close(o[s], want["o"][s], mag["o"][s], F + off, torch.bfloat16, "o")
        _close(c.state, want["state"], mag["state"], F, torch.float32, "state")


@pytest.mark.parametrize("flags,off", TERMS)
@pytest.mark.parametrize("Hq,Hkv,d,cuts,kind,strided", CASES)
def test_backward(Hq, Hkv, d, cuts, kind, strided, flags, off):
    n, m, x, g2, first, dlast, want, mag = _inputs(Hq, Hkv, d, cuts, kind, strided)
    with Store("bf16", Hq, Hkv, d, 2 * m, flags=flags) as c:
        _fill(c.state[:m], first)
        _fill(c.dstate[m:], dlast)
        at = torch.arange(2 * m, dtype=torch.int32, device="cuda")
        grads = [torch.full((n, h, d), 3.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
        B.pkv_lin_attn_bwd(c.lin, *x, *grads, n, g2, B.lin_batch(m, torch.tensor(cuts, device="cuda"), at[:m], at[m:]),
                           torch.cuda.current_stream())
        B.pkv_lin_check(c.lin)
        s, F = slice(cuts[0], cuts[-1]), (d + 224 + n // 64) * 2.0 ** -24
        for name, t in zip(("dq", "dk", "dv"), grads):
            _close(t[s], want[name][s], mag[name][s], F + off, torch.bfloat16, name)
        _close(c.dstate[:m], want["dstate"], mag["dstate"], F, torch.float32, "dstate")


def test_one_term_on_streams_and_in_graphs():
    base.test_graphs_streams_and_repeats("bf16", B.PKV_FLAG_LIN_ONE_TERM)


@pytest.mark.parametrize("dtype,flags", [("f32", 0), ("bf16", B.PKV_FLAG_SIMT_ONLY)])
def test_the_flag_changes_tensor_core_calls_alone(dtype, flags):
    """Calls on the CUDA cores, and single tokens, are the same bits with it."""
    Hq, Hkv, d, n = 4, 2, 64, 200
    q, k, v, do = _rows(n, (Hq, Hkv, Hkv, Hq), d, base.DT[dtype][0], False, 7)
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for extra in (0, B.PKV_FLAG_LIN_ONE_TERM):
        with Store(dtype, Hq, Hkv, d, 1, flags=flags | extra) as c:
            out = [torch.empty_like(t) for t in (q, q, k, v, q[:1])]
            st = torch.cuda.current_stream()
            batch = B.lin_batch(1, None, None, slot)
            B.pkv_lin_attn_fwd(c.lin, q, k, v, out[0], n, None, batch, st)
            B.pkv_lin_attn_bwd(c.lin, q, k, v, do, *out[1:4], n, None, batch, st)
            B.pkv_lin_attn_step(c.lin, q[:1], k[:1], v[:1], out[4], 1, None, slot, st)
            B.pkv_lin_check(c.lin)
            got.append(out + [c.state.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*got))
