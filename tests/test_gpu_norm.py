"""Layer norm against its definition in float64.

Bounds, from the arithmetic; u = 2^-24. A sum over a group adds at most 32
elements in a thread, 5 steps over lanes and 32 warps: 70 u of the sum of absolute
values. The mean is off by 72 u mean|x| (with the division), so x - mean by that
and u |x - mean|; the variance by 72 u + 2 u relative, plus the square of the mean's
error; rstd by half of that and 3 u for root, sum and division: 45 u, times xhat.
The product with w, the sum with b: 2 u each.
dx = rstd (t - m1 - xhat m2) with the statistics given: each of the three terms is
off by at most 80 u of itself or of the mean of absolute values behind it. dw, db: n
additions at most, with the columns' shares: (n + 80) u of the sum of absolute values.
Storage rounds once: half an eps of the type."""
import numpy as np
import pytest
import torch

import lin_oracle as O
from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": (torch.bfloat16, B.PKV_BF16), "f32": (torch.float32, B.PKV_F32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, tol, dt, what):
    half = torch.finfo(dt).eps / 2
    over = np.abs(_f64(got).reshape(want.shape) - want) - (tol + half * (np.abs(want) + tol))
    assert not np.isnan(over).any() and over.max(initial=0) <= 0, (what, over.max(), np.argmax(over))


CASES = [
    # dtype, weights, n, groups, width, gap behind each row, bias, offset of x
    ("bf16", "bf16", 1, 1, 3584, 0, True, 0.0),
    ("bf16", "f32", 5, 1, 8, 0, True, 3.0),
    ("bf16", "bf16", 33, 14, 64, 64, False, 0.0),
    ("bf16", "bf16", 700, 28, 128, 0, True, 1.0),
    ("bf16", "f32", 9, 3, 80, 8, True, 0.0),
    ("bf16", None, 17, 1, 1, 0, False, 0.0),
    ("bf16", "bf16", 65, 1, 1001, 0, True, -2.0),
    ("bf16", "bf16", 40, 2, 257, 3, True, 0.0),
    ("bf16", None, 3, 1, 32768, 0, False, 0.5),
    ("bf16", "bf16", 6, 1, 8200, 0, True, 0.0),
    ("f32", "f32", 1000, 1, 256, 0, True, 0.0),
    ("f32", "bf16", 21, 5, 36, 4, True, 10.0),
    ("f32", None, 4, 1, 7, 1, False, 0.0),
    ("f32", "f32", 12, 1, 4100, 0, True, 0.0),
    ("f32", "f32", 2, 1, 32767, 0, True, 0.0),
    ("f32", "f32", 310, 1, 1024, 0, False, 0.0),
    ("bf16", "f32", 5000, 1, 16, 0, True, 0.0),
    ("bf16", "f32", 70, 2, 5001, 3, True, 0.5),          # wide rows by single elements
    ("bf16", "bf16", 600, 1, 8208, 0, True, 0.0),        # and by vectors, more rows than shares
    ("f32", "f32", 9, 2, 8200, 4, True, 0.0),
    ("f32", None, 30, 3, 4099, 0, False, 1.0),
    ("bf16", "bf16", 3000, 1, 512, 0, True, 0.0),        # many teams a CTA
    ("bf16", "bf16", 4096, 28, 128, 0, True, 0.0),
]


def _inputs(dtype, weights, n, groups, width, gap, bias, offset):
    dt, g = DT[dtype][0], torch.Generator().manual_seed(n + width)
    cols = groups * width
    x = (torch.randn(n, cols + gap, generator=g) + offset).to(dt).cuda()[:, :cols]
    dy = torch.randn(n, cols + gap, generator=g).to(dt).cuda()[:, :cols]
    wt = None if weights is None else DT[weights][0]
    w = None if wt is None else (1 + 0.3 * torch.randn(cols, generator=g)).to(wt).cuda()
    b = None if wt is None or not bias else torch.randn(cols, generator=g).to(wt).cuda()
    return dt, x, dy, w, b


@pytest.mark.parametrize("dtype,weights,n,groups,width,gap,bias,offset", CASES)
def test_forward_and_backward(dtype, weights, n, groups, width, gap, bias, offset):
    dt, x, dy, w, b = _inputs(dtype, weights, n, groups, width, gap, bias, offset)
    cols, shape = groups * width, (n, groups, width)
    m = B.norm(width, groups, 1e-4, w, b, DT[dtype][1])
    y = torch.full((n, cols + gap), 3.0, dtype=dt, device="cuda")
    mean, rstd = (torch.empty(n, groups, device="cuda") for _ in range(2))
    st = torch.cuda.current_stream()
    B.pkv_layer_norm_fwd(x, y[:, :cols], mean, rstd, n, m, st)
    X, D = _f64(x).reshape(shape), _f64(dy).reshape(shape)
    W = np.ones((groups, width)) if w is None else _f64(w).reshape(groups, width)
    Bv = np.zeros((groups, width)) if b is None else _f64(b).reshape(groups, width)
    want, wm, wr = O.norm_forward(X, W, Bv, 1e-4)
    ax = np.abs(X).mean(-1)
    tm = 72 * U * ax
    tr = wr * (45 * U + (tm * wr) ** 2)
    _close(mean, wm, tm, torch.float32, "mean")
    _close(rstd, wr, tr, torch.float32, "rstd")
    xhat = np.abs((X - wm[..., None]) * wr[..., None])
    tol = np.abs(W) * ((tm * wr)[..., None] + xhat * (50 * U + ((tm * wr) ** 2)[..., None])) + 4 * U * (np.abs(W) * xhat + np.abs(Bv))
    _close(y[:, :cols], want, tol, dt, "y")
    assert gap == 0 or (y[:, cols:] == 3.0).all()
    # The backward, from the statistics as the forward gave them.
    fm, fr = _f64(mean), _f64(rstd)
    dx = torch.full((n, cols + gap), 3.0, dtype=dt, device="cuda")
    dw, db = (torch.full((cols,), 2.0, device="cuda") for _ in range(2))
    scratch = torch.full((B.pkv_layer_norm_scratch(m, n) + 4,), 9.0, device="cuda")
    B.pkv_layer_norm_bwd(dy, x, mean, rstd, dx[:, :cols], dw, db, n, m, scratch[:-4], stream=st)
    assert (scratch[-4:] == 9.0).all()
    wx, ww, wb = O.norm_backward(D, X, W, fm, fr)
    H = np.abs((X - fm[..., None]) * fr[..., None])
    u = np.abs(D * W)
    tol = 80 * U * fr[..., None] * (u + u.mean(-1, keepdims=True) + 2 * H * (u * H).mean(-1, keepdims=True))
    _close(dx[:, :cols], wx, tol, dt, "dx")
    assert gap == 0 or (dx[:, cols:] == 3.0).all()
    _close(dw, ww, (n + 80) * U * (np.abs(D) * H).sum(0), torch.float32, "dw")
    _close(db, wb, (n + 80) * U * np.abs(D).sum(0), torch.float32, "db")
    # Added to what is there; each output alone; in place; the same bits.
    again, other = dw.clone(), torch.empty_like(db)
    B.pkv_layer_norm_bwd(dy, x, mean, rstd, None, again, None, n, m, scratch, accumulate=True, stream=st)
    B.pkv_layer_norm_bwd(dy, x, mean, rstd, None, None, other, n, m, scratch, stream=st)
    assert torch.equal(again, dw + dw) and torch.equal(other, db)
    g = dy.clone()
    B.pkv_layer_norm_bwd(g, x, mean, rstd, g, None, None, n, m, None, stream=st)
    z = x.clone()
    B.pkv_layer_norm_fwd(z, z, None, None, n, m, st)
    if gap == 0:                                         # (a row stride may change the kernel's vectors and so the sums' order)
        assert torch.equal(g, dx) and torch.equal(z, y)


def test_no_rows():
    m = B.norm(64)
    e, s = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 1, device="cuda")
    dw, db = torch.full((64,), 2.0, device="cuda"), torch.full((64,), 2.0, device="cuda")
    B.pkv_layer_norm_fwd(e, e, s, s, 0, m)
    B.pkv_layer_norm_bwd(e, e, s, s, e, dw, None, 0, m, None)
    B.pkv_layer_norm_bwd(e, e, s, s, e, None, db, 0, m, None, accumulate=True)
    assert not dw.any() and (db == 2.0).all()


def test_rows_that_are_not_finite_keep_to_themselves():
    n, width = 12, 512
    x = torch.randn(n, width, device="cuda")
    dy = torch.randn_like(x)
    x[3, 5], x[7, 0] = float("nan"), float("inf")
    m = B.norm(width, dtype=B.PKV_F32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(n, 1, device="cuda"), torch.empty(n, 1, device="cuda")
    B.pkv_layer_norm_fwd(x, y, mean, rstd, n, m)
    B.pkv_layer_norm_bwd(dy, x, mean, rstd, dx, None, None, n, m, None)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[3, 7]] = True
    for t in (y, dx):
        assert t[~bad].isfinite().all() and not t[bad].isfinite().any()


@pytest.mark.parametrize("width,groups", [(64, 14), (3584, 1)])
def test_graphs_and_streams(width, groups):
    """Two graphs over one scratch, replayed one after the other, on a stream other than the current one."""
    n, cols = 300, width * groups
    dt = torch.bfloat16
    x, dy = (torch.randn(n, cols, device="cuda").to(dt) for _ in range(2))
    w, b = torch.randn(cols, device="cuda"), torch.randn(cols, device="cuda")
    m = B.norm(width, groups, weight=w, bias=b)
    scratch = torch.empty(B.pkv_layer_norm_scratch(m, n), device="cuda")
    side = torch.cuda.Stream()

    def outs():
        return [torch.empty_like(x), torch.empty(n, groups, device="cuda"), torch.empty(n, groups, device="cuda"), torch.empty_like(x),
                torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")]

    def both(o, stream):
        B.pkv_layer_norm_fwd(x, o[0], o[1], o[2], n, m, stream)
        B.pkv_layer_norm_bwd(dy, x, o[1], o[2], o[3], o[4], o[5], n, m, scratch, stream=stream)

    want = outs()
    both(want, torch.cuda.current_stream())
    torch.cuda.synchronize()
    graphs, got = [], []
    for _ in range(2):
        o, g = outs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(o, side)
        graphs.append(g)
        got.append(o)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


@pytest.mark.parametrize("n,width,groups", [(300, 512, 1), (70, 8208, 1), (200, 64, 14)])
def test_calls_at_once(n, width, groups):
    """Two backward passes on two streams, each with scratch of its own, and two graphs that share
    one replayed in turn: the bits of each by itself."""
    cols = groups * width
    g = torch.Generator().manual_seed(n)
    xs, dys = ([torch.randn(n, cols, generator=g).bfloat16().cuda() for _ in range(2)] for _ in range(2))
    w = torch.randn(cols, generator=g).bfloat16().cuda()
    m = B.norm(width, groups, 1e-5, w, None, B.PKV_BF16)
    stats = [[torch.empty(n, groups, device="cuda") for _ in range(2)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for x, (mean, rstd) in zip(xs, stats):
        B.pkv_layer_norm_fwd(x, torch.empty_like(x), mean, rstd, n, m)
    scratch = [torch.empty(B.pkv_layer_norm_scratch(m, n), device="cuda") for _ in range(2)]

    def outs():
        return [[torch.zeros_like(xs[0]), torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")] for _ in range(2)]

    def run(s, out, sc, stream):
        B.pkv_layer_norm_bwd(dys[s], xs[s], *stats[s], *out, n, m, sc, stream=stream)
    want, got, replayed = outs(), outs(), outs()
    for s in range(2):
        run(s, want[s], scratch[0], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(3):
        for s in range(2):
            run(s, got[s], scratch[s], streams[s])
    torch.cuda.synchronize()
    graphs = []
    for s in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[s], stream=streams[0]):
            run(s, replayed[s], scratch[0], streams[0])
    for s in (0, 1, 0, 1):
        graphs[s].replay()
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[s], want[s])) and all(torch.equal(a, b) for a, b in zip(replayed[s], want[s]))
