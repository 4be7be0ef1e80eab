"""Argument refusals of linear attention and layer norm. No GPU: the store holds
no memory (PKV_RES_META) and the addresses are made up and never read."""
import ctypes

import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build


@pytest.fixture(scope="module")
def lin():
    pkv_build.build()
    h = B.pkv_lin_create(2, 4, 64, B.PKV_BF16, 3, grads=True, residency=B.PKV_RES_META)
    yield h
    B.pkv_lin_destroy(h)


@pytest.mark.parametrize("kw,status", [
    (dict(n_kv_heads=0), B.PKV_ERR_INVALID), (dict(n_q_heads=3), B.PKV_ERR_INVALID), (dict(n_q_heads=0), B.PKV_ERR_INVALID),
    (dict(head_dim=96), B.PKV_ERR_UNSUPPORTED), (dict(dtype=2), B.PKV_ERR_INVALID), (dict(n_slots=0), B.PKV_ERR_INVALID),
    (dict(n_slots=1 << 40), B.PKV_ERR_INVALID), (dict(residency=B.PKV_RES_PINNED_HOST), B.PKV_ERR_INVALID),
    (dict(flags=8), B.PKV_ERR_INVALID), (dict(n_q_heads=70000, n_kv_heads=70000), B.PKV_ERR_UNSUPPORTED),
])
def test_bad_store(lin, kw, status):
    args = dict(n_kv_heads=2, n_q_heads=4, head_dim=64, dtype=B.PKV_BF16, n_slots=3, residency=B.PKV_RES_META)
    with pytest.raises(B.PkvError) as e:
        B.pkv_lin_create(**{**args, **kw})
    assert e.value.status == status


def test_store_without_memory(lin):
    assert B.pkv_lin_arrays(lin) == {"state": None, "dstate": None}
    B.pkv_lin_check(lin)
    B.pkv_lin_destroy(None)
    l = B.lib()
    assert l.pkv_lin_create(None, None) == B.PKV_ERR_INVALID
    assert l.pkv_lin_check(None) == B.PKV_ERR_INVALID and l.pkv_lin_arrays(None, None, None) == B.PKV_ERR_INVALID


def _fwd(lin, n=4, q=64, k=64, v=64, o=64, strides=(0, 0, 0, 0), decay=None, batch=B.lin_batch()):
    p = [x for pair in zip((q, k, v, o), strides) for x in pair]
    return B.lib().pkv_lin_attn_fwd(lin, *p, n, decay, None if batch is None else ctypes.byref(batch), None)


def _bwd(lin, n=4, ptrs=(64,) * 7, strides=(0,) * 7, decay=None, batch=B.lin_batch()):
    p = [x for pair in zip(ptrs, strides) for x in pair]
    return B.lib().pkv_lin_attn_bwd(lin, *p, n, decay, None if batch is None else ctypes.byref(batch), None)


def test_bad_attention_operands(lin):
    bad_batches = (None, B.lin_batch(0), B.lin_batch(2), B.lin_batch(-1, 64), B.lin_batch(1, 68), B.lin_batch(1, 64, 66),
                   B.lin_batch(1, 64, 64, 66))
    for bad in [dict(n=-1), dict(n=1 << 40), dict(decay=66)] + [dict(batch=b) for b in bad_batches]:
        assert _fwd(lin, **bad) == B.PKV_ERR_INVALID, bad
        assert _bwd(lin, **bad) == B.PKV_ERR_INVALID, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=72), dict(k=72), dict(v=68), dict(o=72),
                dict(strides=(255, 0, 0, 0)), dict(strides=(0, 120, 0, 0)), dict(strides=(0, 0, 132, 0)),
                dict(strides=(0, 0, 0, -256))):
        assert _fwd(lin, **bad) == B.PKV_ERR_INVALID, bad
    for i in range(7):
        for wrong in (None, 72):
            assert _bwd(lin, ptrs=tuple(wrong if x == i else 64 for x in range(7))) == B.PKV_ERR_INVALID, i
        assert _bwd(lin, strides=tuple(100 if x == i else 0 for x in range(7))) == B.PKV_ERR_INVALID, i
    for call in (_fwd, _bwd):
        assert call(None) == B.PKV_ERR_INVALID
        assert call(lin) == B.PKV_ERR_INVALID and "META" in B.pkv_last_error()      # every check before it passes
        assert call(lin, batch=B.lin_batch(1 << 30, 64)) == B.PKV_ERR_UNSUPPORTED
    no_grads = B.pkv_lin_create(2, 4, 64, residency=B.PKV_RES_META)
    assert _bwd(no_grads) == B.PKV_ERR_INVALID and "without gradients" in B.pkv_last_error()
    B.pkv_lin_destroy(no_grads)


def test_bad_step_operands(lin):
    l = B.lib()

    def step(n=4, ptrs=(64,) * 4, strides=(0,) * 4, decay=None, slots=64, handle=lin):
        p = [x for pair in zip(ptrs, strides) for x in pair]
        return l.pkv_lin_attn_step(handle, *p, n, decay, slots, None)

    for bad in (dict(handle=None), dict(n=-1), dict(slots=None), dict(slots=66), dict(decay=2), dict(strides=(0, 0, 0, 8))):
        assert step(**bad) == B.PKV_ERR_INVALID, bad
    for i in range(4):
        assert step(ptrs=tuple(None if x == i else 64 for x in range(4))) == B.PKV_ERR_INVALID
    assert step() == B.PKV_ERR_INVALID and "META" in B.pkv_last_error()
    assert step(n=1 << 30) == B.PKV_ERR_UNSUPPORTED


def test_binding_refuses_tensors_it_cannot_describe(lin):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    for bad in (x.transpose(0, 1), x[:, :, ::2], x[:, 0], x[:1].expand(4, 2, 64), x[:3], x.float(), q, x):
        why = "CUDA" if bad is x else ""
        with pytest.raises(ValueError, match=why):
            B.pkv_lin_attn_fwd(lin, 64, bad, 64, 64, 4, None, B.lin_batch())
        with pytest.raises(ValueError, match=why):
            B.pkv_lin_attn_bwd(lin, 64, 64, 64, 64, 64, 64, bad, 4, None, B.lin_batch())
        with pytest.raises(ValueError, match=why):
            B.pkv_lin_attn_step(lin, 64, 64, bad, 64, 4, None, 64)
    i64, i32 = torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    B.lin_batch(2, i64, i32, i32)
    for args in ((2, i32), (3, i64), (2, i64, i64), (2, i64, i32[:1]), (2, i64, None, i64), (2, torch.zeros(6, dtype=torch.int64)[::2])):
        with pytest.raises(ValueError):
            B.lin_batch(*args)
    for batch in (B.lin_batch(2, i64), B.lin_batch(2, 64, i32), B.lin_batch(2, 64, 64, i32)):      # host arrays
        with pytest.raises(ValueError, match="CUDA"):
            B.pkv_lin_attn_fwd(lin, 64, 64, 64, 64, 4, None, batch)
    for decay in (torch.zeros(2), torch.zeros(3), torch.zeros(2, dtype=torch.float64)):
        with pytest.raises(ValueError):
            B.pkv_lin_attn_fwd(lin, 64, 64, 64, 64, 4, decay, B.lin_batch())
    with pytest.raises(ValueError):
        B.pkv_lin_attn_step(lin, 64, 64, 64, 64, 4, None, i32)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), B.PKV_ERR_INVALID), (dict(w_dtype=3), B.PKV_ERR_INVALID), (dict(groups=0), B.PKV_ERR_INVALID),
    (dict(width=0), B.PKV_ERR_INVALID), (dict(width=32769), B.PKV_ERR_UNSUPPORTED), (dict(eps=-1.0), B.PKV_ERR_INVALID),
    (dict(eps=float("nan")), B.PKV_ERR_INVALID), (dict(eps=float("inf")), B.PKV_ERR_INVALID), (dict(weight=65), B.PKV_ERR_INVALID),
    (dict(bias=65), B.PKV_ERR_INVALID),
])
def test_bad_norm(lin, kw, status):
    m = B.norm(64)
    for k, v in kw.items():
        setattr(m, k, v)
    l, f = B.lib(), ctypes.c_int64()
    m = ctypes.byref(m)
    assert l.pkv_layer_norm_fwd(64, 0, 64, 0, None, None, 4, m, None) == status
    assert l.pkv_layer_norm_scratch(m, 4, ctypes.byref(f)) == status
    assert l.pkv_layer_norm_bwd(64, 0, 64, 0, 64, 64, 64, 0, 64, 64, 0, 64, 4, m, None) == status


def test_bad_norm_operands(lin):
    l, m = B.lib(), ctypes.byref(B.norm(64, groups=2))
    for x, xs, y, ys, mean, rstd, n, d in ((None, 0, 64, 0, None, None, 4, m), (64, 0, None, 0, None, None, 4, m),
                                           (65, 0, 64, 0, None, None, 4, m), (64, 127, 64, 0, None, None, 4, m),
                                           (64, 0, 64, -128, None, None, 4, m), (64, 0, 64, 0, 64, None, 4, m),
                                           (64, 0, 64, 0, 66, 66, 4, m), (64, 0, 64, 0, None, None, -1, m),
                                           (64, 0, 64, 0, None, None, 1 << 50, m), (64, 0, 64, 0, None, None, 4, None)):
        assert l.pkv_layer_norm_fwd(x, xs, y, ys, mean, rstd, n, d, None) == B.PKV_ERR_INVALID
    good = [64, 0, 64, 0, 64, 64, 64, 0, 64, 64, 0, 64, 4, m, None]
    for at, wrong in ((0, None), (0, 65), (1, 100), (2, None), (3, 1), (4, None), (5, None), (5, 66), (6, 65), (7, 3), (8, 66),
                      (9, 66), (10, 2), (11, None), (11, 72), (12, -1), (13, None)):
        assert l.pkv_layer_norm_bwd(*[wrong if i == at else x for i, x in enumerate(good)]) == B.PKV_ERR_INVALID, (at, wrong)
    assert l.pkv_layer_norm_fwd(None, 0, None, 0, None, None, 0, m, None) == B.PKV_OK          # no rows: nothing to do
    assert l.pkv_layer_norm_scratch(m, 4, None) == B.PKV_ERR_INVALID
    assert B.pkv_layer_norm_scratch(B.norm(64, groups=2), 0) == 0
    assert B.pkv_layer_norm_scratch(B.norm(64, groups=2), 1) >= 2 * 128


def test_binding_norm_tensors(lin):
    w = torch.ones(128, dtype=torch.bfloat16)
    assert B.norm(64, groups=2, weight=w).w_dtype == B.PKV_BF16
    assert B.norm(64, groups=2, weight=w.float(), bias=w.float()).w_dtype == B.PKV_F32
    for kw in (dict(weight=w[:64]), dict(weight=w, bias=w.float()), dict(weight=w.half()), dict(weight=w, w_dtype=B.PKV_F32)):
        with pytest.raises(ValueError):
            B.norm(64, groups=2, **kw)
    m = B.norm(64, groups=2)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for bad in (x.float(), x[:3], x[:, :64], x.t(), torch.zeros(4, 256, dtype=torch.bfloat16)[:, ::2], x[:1].expand(4, 128), x):
        with pytest.raises(ValueError, match="CUDA" if bad is x else ""):
            B.pkv_layer_norm_fwd(bad, 64, None, None, 4, m)
        with pytest.raises(ValueError, match="CUDA" if bad is x else ""):
            B.pkv_layer_norm_bwd(64, 64, 64, 64, bad, None, None, 4, m, None)
    for bad in (torch.zeros(8), torch.zeros(7), torch.zeros(8, dtype=torch.float64)):
        with pytest.raises(ValueError):
            B.pkv_layer_norm_fwd(64, 64, bad, bad, 4, m)
    with pytest.raises(ValueError, match="scratch"):
        B.pkv_layer_norm_bwd(64, 64, 64, 64, None, 64, None, 4, m, torch.zeros(3))


def test_flags_of_a_store():
    for flags in (0, B.PKV_FLAG_SIMT_ONLY, B.PKV_FLAG_LIN_ONE_TERM, B.PKV_FLAG_SIMT_ONLY | B.PKV_FLAG_LIN_ONE_TERM):
        B.pkv_lin_destroy(B.pkv_lin_create(2, 4, 64, residency=B.PKV_RES_META, flags=flags))
    for flags in (4, 4 | B.PKV_FLAG_LIN_ONE_TERM, 1 << 31):
        with pytest.raises(B.PkvError) as e:
            B.pkv_lin_create(2, 4, 64, residency=B.PKV_RES_META, flags=flags)
        assert e.value.status == B.PKV_ERR_INVALID
