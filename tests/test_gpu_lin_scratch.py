"""The scratch memory of a store of states over calls of rising length: bounded by the longest
call's, though outgrown buffers stay (captured graphs may use them)."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from test_gpu_lin import Store, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,step", [("bf16", 128), ("f32", 64)])
def test_rising_lengths(dtype, step):
    """50 prompts, each a chunk longer than the one before, against the longest alone. With every
    buffer at least twice the one before, the last is less than twice what the longest call needs
    and all together less than twice the last."""
    H, d, most = 16, 128, 50
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.randn(most * step, H, d, device="cuda").to(dt)
    o = torch.empty_like(x)

    def taken(lengths):
        with Store(dtype, H, H, d, 1, grads=False) as c:
            B.pkv_lin_attn_fwd(c.lin, x[:0], x[:0], x[:0], o[:0], 0, None, B.lin_batch(), torch.cuda.current_stream())   # the first buffer
            torch.cuda.synchronize()
            before = torch.cuda.mem_get_info()[0]
            for n in lengths:
                B.pkv_lin_attn_fwd(c.lin, x[:n], x[:n], x[:n], o[:n], n, None, B.lin_batch(), torch.cuda.current_stream())
            torch.cuda.synchronize()
            B.pkv_lin_check(c.lin)
            return before - torch.cuda.mem_get_info()[0]

    alone = taken([most * step])
    assert alone > 0
    rising = taken(range(step, (most + 1) * step, step))
    assert rising <= 4 * alone + (32 << 20), (rising, alone)        # (a page of 2 MB for each of the few buffers)


def test_results_do_not_depend_on_the_scratch():
    """The same bits in a buffer that is just large enough and in one that an earlier call made larger."""
    H, d, n = 4, 64, 500
    x = torch.randn(900, H, d, device="cuda").bfloat16()
    got = []
    for lengths in ([n], [300, 900, n], [n - 1, n]):
        with Store("bf16", H, H, d, 1, grads=False) as c:
            for m in lengths:
                o = torch.empty_like(x[:m])
                B.pkv_lin_attn_fwd(c.lin, x[:m], x[:m], x[:m], o, m, None, B.lin_batch(), torch.cuda.current_stream())
            torch.cuda.synchronize()
            got.append(o)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
