"""Modified scores on staged pools where only the pages that some query sees are
staged: the others' block-table entries are unusable, and no call may want them.
Ranges of neighbouring queries lie apart, so that pages without any visible key
lie between the keys of one tile. Bounds are mod_oracle's."""
import numpy as np
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build
from test_gpu_attn_mod import Case, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _ranges(kind, q_start, n, P):
    i = q_start + np.arange(n)
    lo, hi = i // P * P, i + 1                              # the query's own page
    if kind == "window":                                    # from inside a page on, not a multiple of any tile
        lo = np.maximum(i - 37, 0)
    elif kind == "apart":                                   # every third query sees the first page alone
        far = np.arange(n) % 3 == 1
        lo, hi = np.where(far, 3, lo), np.where(far, min(P, 100), hi)
    elif kind == "tiles":                                   # queries up to 127: the first page; later ones: their own
        far = np.arange(n) < 128
        lo, hi = np.where(far, 0, lo), np.where(far, P - 5, hi)
    return torch.from_numpy(lo), torch.from_numpy(hi)


def _seen(lo, hi, P):
    pages = set()
    for a, b in zip(lo.tolist(), hi.tolist()):
        pages.update(range(a // P, (b - 1) // P + 1) if b > a else ())
    return sorted(pages)


def _run(dtype, Hq, Hkv, d, P, q_start, n, kind, cap=0.0, bias=False, sel=None, missing=None):
    c = Case(dtype, Hq, Hkv, d, P, q_start, n, cap=cap, bias=bias, seed=31, sel=sel)
    pages = -(-c.L // P)
    lo, hi = _ranges(kind, q_start, n, P)
    staged = [p for p in _seen(lo, hi, P) if p != missing]
    assert len(staged) < pages
    pool = B.pkv_pool_create(P, Hkv, Hq, d, B.PKV_BF16 if c.bf16 else B.PKV_F32, pages, residency=B.PKV_RES_PINNED_HOST,
                             n_device_slots=len(staged))
    try:
        seq = B.pkv_seq_create(pool)
        B.pkv_append(seq, c.k, c.v, c.L)
        c.k_begin, c.k_end = lo, hi
        c.mod = B.score_mod(cap, None if c.slopes is None else c.slopes.cuda(), lo.cuda(), hi.cuda())
        B.pkv_prefetch(seq, torch.tensor(staged, dtype=torch.int32, device="cuda"), len(staged), 3)
        B.pkv_wait(seq)
        o, lse = torch.empty(n, Hq, d, dtype=c.dt, device="cuda"), torch.empty(Hq, n, device="cuda")
        dq = torch.empty_like(o)
        B.pkv_chunk_attn_mod_fwd(seq, c.q, q_start, n, o, lse, c.mod, c.sel)
        if missing is not None:
            with pytest.raises(B.PkvError) as e:
                B.pkv_check(pool)
            assert e.value.status == B.PKV_ERR_DEVICE_FAULT and "page index" in str(e.value)
            return
        B.pkv_chunk_attn_mod_bwd(seq, c.q, o, c.dout, lse, q_start, n, dq, c.mod, c.sel)
        B.pkv_writeback_grads(seq)
        dk, dv = (torch.empty(c.L, Hkv, d, device="cuda") for _ in range(2))
        B.pkv_gather(seq, dk=dk, dv=dv)
        B.pkv_check(pool)
        r, tol = c.oracle()
        for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            a, b = _f64(t), r[name]
            inf = np.isinf(b)
            assert np.array_equal(a[inf], b[inf]), name
            assert (np.abs(a - b)[~inf] <= tol[name][~inf]).all(), name
    finally:
        B.pkv_pool_destroy(pool)
        c.close()


@pytest.mark.parametrize("kind", ["window", "apart", "own"])
@pytest.mark.parametrize("dtype,Hq,Hkv,d,P,q_start,n", [
    ("bf16", 6, 2, 64, 32, 333, 1), ("bf16", 28, 4, 128, 16, 410, 3), ("bf16", 10, 1, 64, 48, 500, 13),
    ("bf16", 5, 1, 128, 128, 700, 16)])
def test_few_queries(dtype, Hq, Hkv, d, P, q_start, n, kind):
    _run(dtype, Hq, Hkv, d, P, q_start, n, kind, cap=20.0, bias=True)


@pytest.mark.parametrize("kind", ["window", "apart", "tiles"])
@pytest.mark.parametrize("Hq,Hkv,d,n", [(7, 1, 128, 256), (6, 2, 64, 300), (3, 1, 64, 100), (28, 4, 128, 257)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True)])
def test_tensor_core_tiles(Hq, Hkv, d, n, kind, cap, bias):
    _run("bf16", Hq, Hkv, d, 128, 640, n, kind, cap=cap, bias=bias)


@pytest.mark.parametrize("kind", ["window", "apart", "tiles"])
@pytest.mark.parametrize("dtype,P,n", [("bf16", 32, 40), ("bf16", 16, 150), ("f32", 16, 70), ("f32", 128, 140)])
def test_cuda_core_tiles(dtype, P, n, kind):
    _run(dtype, 6, 2, 64, P, 6 * 128, n, kind, cap=8.0, bias=True)


@pytest.mark.parametrize("dtype,P,n", [("bf16", 128, 200), ("f32", 16, 50)])
def test_listed_pages_that_no_query_sees(dtype, P, n):
    """A selection lists pages that the ranges hide: those need no slot either."""
    _run(dtype, 4, 2, 64, P, 5 * P, n, "own", cap=8.0, sel=3)


@pytest.mark.parametrize("dtype,Hq,Hkv,d,P,n", [("bf16", 6, 2, 64, 32, 5), ("bf16", 7, 1, 128, 128, 256), ("f32", 4, 2, 64, 16, 40)])
def test_a_seen_page_that_is_not_staged_is_an_error(dtype, Hq, Hkv, d, P, n):
    _run(dtype, Hq, Hkv, d, P, 640, n, "apart", missing=0)
