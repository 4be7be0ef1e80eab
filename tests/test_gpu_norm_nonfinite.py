"""Rows with a NaN or an infinity, in every kernel of the layer norm: they keep to their own row and
group, and dw and db to their columns."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from test_gpu_norm import DT, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n,groups,width", [
    ("bf16", 40, 14, 64), ("bf16", 12, 28, 128), ("f32", 30, 3, 5), ("bf16", 9, 1, 24), ("bf16", 12, 1, 512), ("bf16", 12, 2, 3584),
    ("f32", 12, 2, 1001), ("bf16", 12, 1, 8208), ("bf16", 12, 2, 5001), ("f32", 12, 1, 8200), ("f32", 12, 1, 32767),
])
def test_bad_rows_keep_to_themselves(dtype, n, groups, width):
    dt, kind = DT[dtype]
    cols = groups * width
    gen = torch.Generator().manual_seed(width)
    x, dy = (torch.randn(n, cols, generator=gen).to(dt).cuda() for _ in range(2))
    w = torch.randn(cols, generator=gen).cuda()
    m = B.norm(width, groups, 1e-5, w, w, kind)
    scratch = torch.empty(B.pkv_layer_norm_scratch(m, n), device="cuda")
    got = []
    for bad in (False, True):
        z, u = x.clone(), dy.clone()
        if bad:
            z[3, 2], z[7, width - 1], u[5, 1] = float("nan"), float("inf"), float("nan")
        y, dx = torch.empty_like(z), torch.empty_like(z)
        mean, rstd = (torch.empty(n, groups, device="cuda") for _ in range(2))
        dw, db = (torch.empty(cols, device="cuda") for _ in range(2))
        B.pkv_layer_norm_fwd(z, y, mean, rstd, n, m, torch.cuda.current_stream())
        B.pkv_layer_norm_bwd(u, z, mean, rstd, dx, dw, db, n, m, scratch, stream=torch.cuda.current_stream())
        got.append([t.reshape(n, groups, width) for t in (y, dx)] + [dw, db])
    (y0, dx0, dw0, db0), (y1, dx1, dw1, db1) = got
    for a, b, rows in ((y0, y1, [3, 7]), (dx0, dx1, [3, 5, 7])):
        hit = torch.zeros(n, groups, dtype=torch.bool, device="cuda")
        hit[rows, 0] = True
        assert torch.equal(a[~hit], b[~hit]) and not b[hit].isfinite().any()
    assert torch.equal(dw0[width:], dw1[width:]) and not dw1[:width].isfinite().any()
    same = torch.ones(cols, dtype=torch.bool, device="cuda")
    same[1] = False
    assert torch.equal(db0[same], db1[same]) and db1[1].isnan()
