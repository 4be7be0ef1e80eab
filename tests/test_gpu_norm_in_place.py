"""Layer norm's backward with dx in dy's memory: the bits of the call into other memory, of
dx, dw and db together, whichever kernels the width, the strides and the addresses choose."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from test_gpu_norm import CASES, DT, _inputs, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _check(x, dy, w, b, groups, width, dtype, place):
    """place(): new rows for gradients; dy's are given there, so that strides and addresses are the same."""
    n, cols = x.shape
    m = B.norm(width, groups, 1e-4, w, b, DT[dtype][1])
    st = torch.cuda.current_stream()
    mean, rstd = (torch.empty(n, groups, device="cuda") for _ in range(2))
    B.pkv_layer_norm_fwd(x, torch.empty_like(x), mean, rstd, n, m, st)
    scratch = torch.empty(B.pkv_layer_norm_scratch(m, n), device="cuda")
    apart, into = place(), place()
    into.copy_(dy)
    dw, db, dw_in, db_in = (torch.full((cols,), 2.0, device="cuda") for _ in range(4))
    B.pkv_layer_norm_bwd(dy, x, mean, rstd, apart, dw, db, n, m, scratch, stream=st)
    B.pkv_layer_norm_bwd(into, x, mean, rstd, into, dw_in, db_in, n, m, scratch, stream=st)
    for name, want, got in (("dx", apart, into), ("dw", dw, dw_in), ("db", db, db_in)):
        assert torch.equal(want, got), name


@pytest.mark.parametrize("dtype,weights,n,groups,width,gap,bias,offset", CASES)
def test_backward_in_place(dtype, weights, n, groups, width, gap, bias, offset):
    _, x, dy, w, b = _inputs(dtype, weights, n, groups, width, gap, bias, offset)
    cols = groups * width
    _check(x, dy, w, b, groups, width, dtype, lambda: torch.zeros(n, cols + gap, dtype=x.dtype, device="cuda")[:, :cols])


@pytest.mark.parametrize("dtype,n,width", [("bf16", 50, 4104), ("f32", 21, 8192), ("bf16", 7, 32768), ("bf16", 40, 512)])
def test_backward_in_place_at_an_odd_address(dtype, n, width):
    """Rows of whole vectors that do not start at one: read by single elements, wide ones by the wide kernels."""
    _, x, dy, w, b = _inputs(dtype, "f32", n, 1, width, 0, True, 0.5)

    def place():
        return torch.zeros(n, width + 8, dtype=x.dtype, device="cuda")[:, 1:1 + width]
    at = [place().copy_(t) for t in (x, dy)]
    _check(*at, w, b, 1, width, dtype, place)
