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


def _captured_append(s, kb, vb, n, side):
    """The append in a graph, with K and V gathered behind it."""
    a, b = torch.empty_like(kb), torch.empty_like(vb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.pkv_append(s, kb, vb, n, side)
        B.pkv_gather(s, a, b, stream=side)
    return g, a, b


def test_append_captured_after_a_reset():
    """The graph holds an upload of its own: replays store new rows into the same
    pages, also after other appends of the sequence have run."""
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 8)
    try:
        s, side = B.pkv_seq_create(pool), torch.cuda.Stream()
        k, v = _rows(60, 1)
        B.pkv_append(s, k, v, 60, torch.cuda.current_stream())
        torch.cuda.synchronize()
        B.pkv_seq_reset(s)
        kb, vb = k.clone(), v.clone()
        g, a, b = _captured_append(s, kb, vb, 60, side)
        assert B.pkv_seq_length(s) == 60
        for seed in (2, 3):
            k, v = _rows(60, seed)
            kb.copy_(k), vb.copy_(v)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, k) and torch.equal(b, v) and _holds(s, k, v)
            B.pkv_seq_reset(s)                               # the same pages, without the graph
            k, v = _rows(60, 10 + seed)
            B.pkv_append(s, k, v, 60, torch.cuda.current_stream())
            assert _holds(s, k, v)
            torch.cuda.synchronize()
        B.pkv_check(pool)
    finally:
        B.pkv_pool_destroy(pool)


def test_a_captured_upload_counts_only_where_it_runs():
    """A first append that was captured and never replayed has sent nothing."""
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 8)
    try:
        s, side = B.pkv_seq_create(pool), torch.cuda.Stream()
        k, v = _rows(60, 4)
        kb, vb = k.clone(), v.clone()
        torch.cuda.synchronize()
        g, a, b = _captured_append(s, kb, vb, 60, side)
        B.pkv_seq_reset(s)
        B.pkv_append(s, k, v, 60, torch.cuda.current_stream())
        assert _holds(s, k, v)
        k, v = _rows(30, 5)
        B.pkv_append(s, k, v, 30, torch.cuda.current_stream())
        torch.cuda.synchronize()
        B.pkv_check(pool)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, kb) and torch.equal(b, vb)
        B.pkv_check(pool)
    finally:
        B.pkv_pool_destroy(pool)


def test_append_captured_with_other_pages_than_before():
    """Entries that were sent change while the stream is being captured."""
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 8)
    try:
        s, t, side = B.pkv_seq_create(pool), B.pkv_seq_create(pool), torch.cuda.Stream()
        st = torch.cuda.current_stream()
        k, v = _rows(60, 6)
        B.pkv_append(s, k, v, 60, st)
        B.pkv_seq_reset(s)
        kt, vt = _rows(30, 7)
        B.pkv_append(t, kt, vt, 30, st)                      # takes pages 0 and 1
        torch.cuda.synchronize()
        g, a, b = _captured_append(s, k, v, 60, side)
        assert B.pkv_get_block_table(s) == [2, 3, 4, 5]
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, k) and torch.equal(b, v)
            assert _holds(s, k, v) and _holds(t, kt, vt)
        k2, v2 = _rows(20, 8)
        B.pkv_append(s, k2, v2, 20, st)                      # goes on behind the captured rows
        assert _holds(s, torch.cat([k, k2]), torch.cat([v, v2]))
        B.pkv_check(pool)
    finally:
        B.pkv_pool_destroy(pool)


def test_append_to_a_pinned_pool_refuses_a_capture():
    """Staging waits for the last append, which a captured one would never be: the
    call claims nothing, and the capture and the sequence go on."""
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 8, residency=B.PKV_RES_PINNED_HOST, n_device_slots=4)
    try:
        s, side = B.pkv_seq_create(pool), torch.cuda.Stream()
        k, v = _rows(60, 1)
        x, y = torch.zeros(4, device="cuda"), torch.ones(4, device="cuda")
        torch.cuda.synchronize()
        g, why = torch.cuda.CUDAGraph(), None
        with torch.cuda.graph(g, stream=side):
            try:
                B.pkv_append(s, k, v, 60, side)
            except B.PkvError as e:
                why = e
            x.add_(y)
        length, free = B.pkv_seq_length(s), B.pkv_pool_free_pages(pool)
        g.replay()
        if not length:
            B.pkv_append(s, k, v, 60, torch.cuda.current_stream())
        B.pkv_prefetch(s, None, 0, 1, torch.cuda.current_stream())
        B.pkv_wait(s, torch.cuda.current_stream())
        assert _holds(s, k, v) and x.eq(1).all()
        B.pkv_check(pool)
        assert why is not None and why.status == B.PKV_ERR_INVALID and "captured" in str(why)
        assert length == 0 and free == 8
    finally:
        B.pkv_pool_destroy(pool)
