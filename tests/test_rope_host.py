"""Argument refusals of the rotation calls, on a pool without page memory:
nothing here reaches a GPU (addresses are made up and never read)."""
import ctypes

import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build


@pytest.fixture(scope="module")
def seq():
    pkv_build.build()
    pool = B.pkv_pool_create(16, 2, 4, 64, B.PKV_BF16, 8, residency=B.PKV_RES_META)
    s = B.pkv_seq_create(pool)
    s_pool = (pool, s)
    yield s_pool
    B.pkv_pool_destroy(pool)


def _rope(**kw):
    r = B.pkv_rope(64, None, 0, 64, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _append(seq, r, n=4, q=None, q_out=None, k=64, v=64, strides=(0, 0, 0)):
    l = B.lib()
    return l.pkv_append_rope(seq, q, strides[0], q_out, k, strides[1], v, strides[2], n,
                             None if r is None else ctypes.byref(r), None)


@pytest.mark.parametrize("kw,status,why", [
    (dict(inv_freq=None), B.PKV_ERR_INVALID, "inv_freq"),
    (dict(rotary_dim=0), B.PKV_ERR_INVALID, "rotary_dim"),
    (dict(rotary_dim=65), B.PKV_ERR_INVALID, "rotary_dim"),
    (dict(rotary_dim=80), B.PKV_ERR_INVALID, "rotary_dim"),
    (dict(rotary_dim=33), B.PKV_ERR_INVALID, "rotary_dim"),
    (dict(rotary_dim=-16), B.PKV_ERR_INVALID, "rotary_dim"),
    (dict(rotary_dim=24), B.PKV_ERR_UNSUPPORTED, "multiple of 16"),
    (dict(interleaved=2), B.PKV_ERR_INVALID, "interleaved"),
    (dict(inv_freq=66), B.PKV_ERR_INVALID, "misaligned"),
    (dict(positions=68), B.PKV_ERR_INVALID, "misaligned"),
])
def test_bad_rotation(seq, kw, status, why):
    pool, s = seq
    r = _rope(**kw)
    l = B.lib()
    assert _append(s, r) == status and why in B.pkv_last_error()
    assert l.pkv_rope_rows(pool, 64, 0, 64, 0, 4, 2, ctypes.byref(r), 0, None) == status
    assert why in B.pkv_last_error()
    assert l.pkv_rope_grad(s, 0, 0, ctypes.byref(r), None, 0, None, 0, None, 0, None, 0, None) == status
    assert why in B.pkv_last_error()


def test_bad_append_operands(seq):
    _, s = seq
    r = _rope()
    for bad in (dict(r=None), dict(r=r, n=-1), dict(r=r, k=None), dict(r=r, v=None), dict(r=r, q=64),
                dict(r=r, q_out=64), dict(r=r, k=72), dict(r=r, v=72), dict(r=r, q=72, q_out=64),
                dict(r=r, q=64, q_out=72), dict(r=r, strides=(0, 127, 0)), dict(r=r, strides=(0, 64, 0)),
                dict(r=r, strides=(0, 0, 132)), dict(r=r, strides=(0, -256, 0)),
                dict(r=r, q=64, q_out=64, strides=(248, 0, 0)), dict(r=r, n=1 << 40)):
        rr = bad.pop("r")
        assert _append(s, rr, **bad) == B.PKV_ERR_INVALID, bad
        assert B.pkv_last_error()
    assert _append(s, r) == B.PKV_ERR_INVALID and "META" in B.pkv_last_error()
    assert _append(s, r, n=0) == B.PKV_OK
    assert B.pkv_seq_length(s) == 0
    assert B.lib().pkv_append_rope(None, None, 0, None, 64, 0, 64, 0, 4, ctypes.byref(r), None) == B.PKV_ERR_INVALID


def test_bad_rows_and_gradient_operands(seq):
    pool, s = seq
    l, r = B.lib(), ctypes.byref(_rope())
    for args in ((None, 64, 0, 64, 0, 4, 2, r, 0, None), (pool, None, 0, 64, 0, 4, 2, r, 0, None),
                 (pool, 64, 0, None, 0, 4, 2, r, 0, None), (pool, 64, 0, 64, 0, -1, 2, r, 0, None),
                 (pool, 64, 0, 64, 0, 4, 0, r, 0, None), (pool, 64, 0, 64, 0, 4, 2, r, 2, None),
                 (pool, 64, 0, 64, 0, 4, 2, None, 0, None), (pool, 64, 100, 64, 0, 4, 2, r, 0, None),
                 (pool, 64, 0, 68, 0, 4, 2, r, 0, None), (pool, 64, 0, 64, 0, 4, 2, r, 0, None)):
        assert l.pkv_rope_rows(*args) == B.PKV_ERR_INVALID, args
    assert "META" in B.pkv_last_error()
    assert l.pkv_rope_grad(None, 0, 0, r, None, 0, None, 0, None, 0, None, 0, None) == B.PKV_ERR_INVALID
    for row0, n in ((-1, 1), (0, 1), (1, 0), (0, -1), (1 << 62, 1 << 62)):
        assert l.pkv_rope_grad(s, row0, n, r, None, 0, None, 0, None, 0, None, 0, None) == B.PKV_ERR_INVALID
    assert l.pkv_rope_grad(s, 0, 0, r, 64, 0, None, 0, None, 0, None, 0, None) == B.PKV_ERR_INVALID


def test_binding_refuses_tensors_it_cannot_describe(seq):
    """Shapes, strides, types and places that the pool's kernels would misread."""
    pool, s = seq
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    inv = torch.ones(32)
    r = B.rope(inv)
    assert r.rotary_dim == 64 and r.interleaved == 0
    for bad in (x.transpose(0, 1), x[:, :, ::2], x[:, 0], x[:1].expand(4, 2, 64), x[:3], x.float(),
                torch.zeros(4, 3, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 32, dtype=torch.bfloat16), x):
        why = "CUDA" if bad is x else ""
        with pytest.raises(ValueError, match=why):
            B.pkv_append_rope(s, None, None, bad, bad, 4, r)
        with pytest.raises(ValueError, match=why):
            B.pkv_rope_rows(pool, bad, bad, 4, 2, r)
        with pytest.raises(ValueError, match=why):
            B.pkv_rope_grad(s, 0, 4, r, dk_out=bad)
    for bad in (inv.double(), torch.ones(64)[::2]):
        with pytest.raises(ValueError):
            B.rope(bad)
    with pytest.raises(ValueError):
        B.rope(inv, positions=torch.zeros(4))
    for r in (B.rope(inv), B.rope(inv, positions=torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(ValueError):                      # the rotation's own arrays
            B.pkv_append_rope(s, None, None, 64, 64, 4, r)
    assert B.rows_ptr(torch.zeros(4, 8, 64)[:, 2:5], 4)[1] == 512
    assert B.rows_ptr(torch.zeros(1, 8, 64)[:, 2:5], 1)[1] == 0


def test_rotation_from_addresses(seq):
    """inv_freq and positions as addresses, like every other operand of the binding."""
    pool, s = seq
    r = B.rope(1 << 20, pos0=7, positions=1 << 21, rotary_dim=32)
    assert (r.inv_freq, r.positions, r.pos0, r.rotary_dim, r.interleaved) == (1 << 20, 1 << 21, 7, 32, 0)
    with pytest.raises(B.PkvError, match="META"):             # every check before the pool's passes
        B.pkv_rope_rows(pool, 64, 64, 4, 2, r)
    inv = torch.ones(32)
    assert B.rope(inv, rotary_dim=64).rotary_dim == 64
    for bad in (lambda: B.rope(1 << 20), lambda: B.rope(None), lambda: B.rope(inv, rotary_dim=32)):
        with pytest.raises(ValueError, match="inv_freq"):
            bad()
    with pytest.raises(B.PkvError, match="rotary_dim"):
        B.pkv_rope_rows(pool, 64, 64, 4, 2, B.rope(1 << 20, rotary_dim=80))
