"""Argument refusals of the attention with modified scores, on a pool without
page memory: nothing here reaches a GPU."""
import ctypes

import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build


@pytest.fixture(scope="module")
def seq():
    pkv_build.build()
    pool = B.pkv_pool_create(16, 2, 4, 64, B.PKV_BF16, 8, residency=B.PKV_RES_META)
    yield B.pkv_seq_create(pool)
    B.pkv_pool_destroy(pool)


def _both(seq, mod, q=64, q_start=0, n=0, sel=None):
    l, m = B.lib(), None if mod is None else ctypes.byref(mod)
    a = l.pkv_chunk_attn_mod_fwd(seq, q, q_start, n, 64, 64, m, sel, None)
    why = B.pkv_last_error()
    b = l.pkv_chunk_attn_mod_bwd(seq, q, 64, 64, 64, q_start, n, 64, m, sel, None)
    assert a == b and why.split(": ", 1)[1] == B.pkv_last_error().split(": ", 1)[1]
    return a, why


@pytest.mark.parametrize("kw,why", [
    (dict(softcap=-1.0), "softcap"), (dict(softcap=float("nan")), "softcap"), (dict(softcap=float("inf")), "softcap"),
    (dict(softcap=1e-4), "softcap"), (dict(softcap=2e4), "softcap"), (dict(slopes=66), "misaligned"),
    (dict(k_begin=68), "misaligned"), (dict(k_end=68), "misaligned"),
])
def test_bad_modification(seq, kw, why):
    m = B.score_mod()
    for k, v in kw.items():
        setattr(m, k, v)
    st, msg = _both(seq, m)
    assert st == B.PKV_ERR_INVALID and why in msg


def test_bad_calls(seq):
    m = B.score_mod(30.0)
    assert _both(seq, None)[0] == B.PKV_ERR_INVALID
    assert _both(None, m)[0] == B.PKV_ERR_INVALID
    for q_start, n in ((-1, 0), (0, -1), (0, 1), (1, 0), (1 << 62, 1 << 62)):
        assert _both(seq, m, q_start=q_start, n=n)[0] == B.PKV_ERR_INVALID, (q_start, n)
    assert _both(seq, m)[0] == B.PKV_OK                     # an empty chunk is no error


def test_binding_checks_the_arrays(seq):
    with pytest.raises(ValueError):
        B.score_mod(slopes=torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        B.score_mod(k_begin=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.score_mod(k_end=torch.zeros(8, dtype=torch.int64)[::2])
    q, lse = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 4)
    for bad in (q.float(), q[:3], q[:, :2], q[:, :, :32], q.transpose(0, 1), q):     # the last: not on a GPU
        with pytest.raises(ValueError):
            B.pkv_chunk_attn_mod_fwd(seq, bad, 0, 4, 64, 64, B.score_mod())
        with pytest.raises(ValueError):
            B.pkv_chunk_attn_mod_bwd(seq, 64, 64, bad, 64, 0, 4, 64, B.score_mod())
    for bad in (lse.double(), lse[:, :3], lse):
        with pytest.raises(ValueError):
            B.pkv_chunk_attn_mod_fwd(seq, 64, 0, 4, 64, bad, B.score_mod())
    for m in (B.score_mod(k_begin=torch.zeros(3, dtype=torch.int64)), B.score_mod(slopes=torch.zeros(5)),
              B.score_mod(k_end=torch.zeros(4, dtype=torch.int64))):
        with pytest.raises(ValueError):
            B.pkv_chunk_attn_mod_fwd(seq, 64, 0, 4, 64, 64, m)
        with pytest.raises(ValueError):
            B.pkv_chunk_attn_mod_bwd(seq, 64, 64, 64, 64, 0, 4, 64, m)


@pytest.mark.parametrize("stream", [None, 1 << 20])
def test_binding_refuses_another_gpus_tensors_without_a_stream_object(monkeypatch, stream):
    """A call without a stream, or with a raw handle, runs on the current device:
    a tensor on another GPU is refused, one on the current GPU is not."""
    class Stand:                                            # a tensor on GPU 1, without a GPU
        device = torch.device("cuda", 1)

        def get_device(self):
            return 1

    dev = B._device(stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        B._on_device(Stand(), dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    B._on_device(Stand(), dev)


def test_binding_checks_the_selection(seq):
    """Its entries are read as int32 [query pages, Hkv, kmax] on the GPU."""
    good = torch.zeros(1, 2, 3, dtype=torch.int32)
    for bad, why in ((good.long(), "int32"), (good[:, :1], "sel must be"), (good[0], "sel must be"),
                     (good.float(), "int32"), (good, "CUDA")):
        with pytest.raises(ValueError, match=why):
            B.pkv_chunk_attn_mod_fwd(seq, 64, 0, 4, 64, 64, B.score_mod(), bad)
        with pytest.raises(ValueError, match=why):
            B.pkv_chunk_attn_mod_bwd(seq, 64, 64, 64, 64, 0, 4, 64, B.score_mod(), bad)
