"""The device copy of the block table: entries a reset sequence gets back are not
sent again, entries that changed or were only reserved are."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(n, 1, 64, generator=g).cuda() for _ in range(2))


def _holds(seq, k, v):
    a, b = torch.empty_like(k), torch.empty_like(v)
    B.pkv_gather(seq, a, b, stream=torch.cuda.current_stream())
    return torch.equal(a, k) and torch.equal(b, v)


def test_reset_sequences_with_the_same_and_with_other_pages():
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 8)
    try:
        s, t = B.pkv_seq_create(pool), B.pkv_seq_create(pool)
        st = torch.cuda.current_stream()
        for turn in range(3):                                # the same pages again and again
            k, v = _rows(60 - turn, turn)
            B.pkv_seq_reset(s)
            B.pkv_append(s, k, v, len(k), st)
            assert B.pkv_get_block_table(s) == [0, 1, 2, 3] and _holds(s, k, v)
        B.pkv_seq_reset(s)
        kt, vt = _rows(40, 7)
        B.pkv_append(t, kt, vt, 40, st)                      # takes pages 0..2
        k, v = _rows(70, 8)
        B.pkv_append(s, k, v, 70, st)
        assert B.pkv_get_block_table(s) == [3, 4, 5, 6, 7]
        assert _holds(s, k, v) and _holds(t, kt, vt)
        B.pkv_seq_reset(t)
        B.pkv_seq_reset(s)
        B.pkv_set_block_table(s, [6, 1, 7])                  # an order of the caller's, then the pool's again
        k, v = _rows(48, 9)
        B.pkv_append(s, k, v, 48, st)
        assert _holds(s, k, v)
        B.pkv_seq_reset(s)
        k, v = _rows(33, 10)
        B.pkv_append(s, k, v, 33, st)
        assert _holds(s, k, v)
        B.pkv_check(pool)
    finally:
        B.pkv_pool_destroy(pool)


def test_reserved_pages_and_another_stream():
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 8)
    try:
        s = B.pkv_seq_create(pool)
        B.pkv_seq_reserve(s, 100)                            # claimed, not sent
        k, v = _rows(90, 1)
        B.pkv_append(s, k[:50], v[:50], 50, torch.cuda.current_stream())
        B.pkv_append(s, k[50:], v[50:], 40, torch.cuda.current_stream())
        assert _holds(s, k, v)
        side = torch.cuda.Stream()
        for seed in range(4):                                # reset, then the next step on the other stream
            torch.cuda.synchronize()
            k, v = _rows(90, 2 + seed)
            stream = side if seed % 2 else torch.cuda.current_stream()
            side.wait_stream(torch.cuda.current_stream())
            B.pkv_seq_reset(s)
            with torch.cuda.stream(stream):
                B.pkv_append(s, k, v, 90, stream)
                assert _holds(s, k, v)
        torch.cuda.synchronize()
        B.pkv_check(pool)
    finally:
        B.pkv_pool_destroy(pool)
