"""Attention with modified scores (cap, distance bias, key ranges) against the
float64 oracle, forward and backward, through the C ABI. Tolerances are the
rounding bounds that mod_oracle.bounds derives, element by element."""
import numpy as np
import pytest
import torch

import mod_oracle
from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs of one call, a pool that holds the keys in permuted pages, and the oracle's answer."""

    def __init__(self, dtype, Hq, Hkv, d, P, q_start, n, extra=0, cap=0.0, bias=False, mask="causal", seed=0, q_scale=1.0,
                 flags=0, sel=None):
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.bf16, self.P, self.q_start, self.n, self.d, self.Hq, self.Hkv = dtype == "bf16", P, q_start, n, d, Hq, Hkv
        self.L = q_start + n + extra
        g = torch.Generator().manual_seed(seed)
        mk = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q = (mk(n, Hq, d) * q_scale).to(self.dt).cuda()
        self.k, self.v = mk(self.L, Hkv, d).to(self.dt).cuda(), mk(self.L, Hkv, d).to(self.dt).cuda()
        self.dout = mk(n, Hq, d).to(self.dt).cuda()
        self.cap, self.slopes = cap, None
        if bias:
            self.slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])
        self.k_begin, self.k_end = self._ranges(mask, np.random.default_rng(seed + 1))
        self.sel, self.listed = None, None
        if sel is not None:
            self._select(sel, np.random.default_rng(seed + 2))
        pages = -(-self.L // P)
        self.pool = B.pkv_pool_create(P, Hkv, Hq, d, B.PKV_BF16 if self.bf16 else B.PKV_F32, pages + 2, flags=flags)
        self.seq = B.pkv_seq_create(self.pool)
        order = np.random.default_rng(seed).permutation(pages + 2)[:pages]
        B.pkv_set_block_table(self.seq, order.tolist())
        B.pkv_append(self.seq, self.k, self.v, self.L, torch.cuda.current_stream())
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.mod = B.score_mod(cap, dev(self.slopes), dev(self.k_begin), dev(self.k_end))

    def _ranges(self, mask, r):
        n, i, L = self.n, self.q_start + np.arange(self.n), self.L
        lo, hi = np.zeros(n, dtype=np.int64), i + 1
        if mask == "causal":
            return None, None
        if mask == "docs":
            cuts = np.unique(np.concatenate([[0], r.integers(0, L, 4)]))
            lo = cuts[np.searchsorted(cuts, i, side="right") - 1]
        elif mask == "window":
            return torch.from_numpy(np.maximum(i + 1 - max(1, L // 3), -5)), None
        elif mask == "prefix":
            return None, torch.from_numpy(np.maximum(hi, self.q_start + n // 2))
        elif mask == "future":                               # keys behind the chunk, beyond the length: clipped
            hi = i + 40
        elif mask == "random":                               # any order, empty rows among them
            lo, hi = r.integers(-10, L, n), r.integers(0, L + 10, n)
        elif mask == "pad":                                  # the last rows and one in the middle see nothing
            hi = hi.copy()
            hi[n - max(1, n // 4):] = 0
            hi[n // 2] = 0
        elif mask == "empty":
            hi = np.zeros(n, dtype=np.int64)
        elif mask == "one":                                  # each query its own key alone
            lo = i.copy()
        return torch.from_numpy(np.ascontiguousarray(lo)), torch.from_numpy(np.ascontiguousarray(hi))

    def _select(self, k, r):
        """Random page lists in the format of pkv_page_topk: ascending, own page last."""
        n_qp = -(-self.n // self.P)
        pages = np.full((n_qp, self.Hkv, k + 1), -1, dtype=np.int32)
        self.listed = np.zeros((self.n, self.Hkv, self.L), dtype=bool)
        for qp in range(n_qp):
            own = self.q_start // self.P + qp
            for h in range(self.Hkv):
                some = sorted(r.permutation(own)[:min(k, own)].tolist()) + [own]
                pages[qp, h, :len(some)] = some
                for p in some:
                    self.listed[qp * self.P:(qp + 1) * self.P, h, p * self.P:(p + 1) * self.P] = True
        self.sel = torch.from_numpy(pages).cuda()

    def kw(self):
        np_ = lambda t: None if t is None else t.numpy().astype(np.float64 if t.is_floating_point() else np.int64)  # noqa: E731
        return dict(cap=self.cap, slopes=np_(self.slopes), k_begin=np_(self.k_begin), k_end=np_(self.k_end), listed=self.listed)

    def oracle(self):
        x = [_f64(t) for t in (self.q, self.k, self.v)]
        r = mod_oracle.attention(*x, self.q_start, dout=_f64(self.dout), **self.kw())
        return r, mod_oracle.bounds(r, *x, self.q_start, self.bf16, dout=_f64(self.dout), **self.kw())

    def forward(self, stream=None):
        o = torch.full((self.n, self.Hq, self.d), 7.0, dtype=self.dt, device="cuda")
        lse = torch.full((self.Hq, self.n), 7.0, device="cuda")
        B.pkv_chunk_attn_mod_fwd(self.seq, self.q, self.q_start, self.n, o, lse, self.mod, self.sel,
                                 stream or torch.cuda.current_stream())
        return o, lse

    def backward(self, o, lse, stream=None):
        dq = torch.full_like(o, 7.0)
        B.pkv_chunk_attn_mod_bwd(self.seq, self.q, o, self.dout, lse, self.q_start, self.n, dq, self.mod, self.sel,
                                 stream or torch.cuda.current_stream())
        return dq

    def grads(self):
        dk, dv = (torch.empty(self.L, self.Hkv, self.d, device="cuda") for _ in range(2))
        B.pkv_gather(self.seq, dk=dk, dv=dv, stream=torch.cuda.current_stream())
        return dk, dv

    def check(self):
        try:
            r, tol = self.oracle()
            o, lse = self.forward()
            dq = self.backward(o, lse)
            dk, dv = self.grads()
            B.pkv_check(self.pool)
            got = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
            worst = {}
            for name, t in got.items():
                a, b = _f64(t), r[name]
                inf = np.isinf(b)
                assert np.array_equal(a[inf], b[inf]), name
                assert np.isfinite(a[~inf]).all(), name
                worst[name] = float((np.abs(a - b)[~inf] / tol[name][~inf]).max(initial=0.0))
            assert max(worst.values()) <= 1.0, worst
            return worst
        finally:
            self.close()

    def close(self):
        if self.pool:
            torch.cuda.synchronize()
            B.pkv_pool_destroy(self.pool)
            self.pool = 0


MASKS = ["causal", "docs", "window", "prefix", "future", "random", "pad", "empty", "one"]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype,P", [("bf16", 128), ("f32", 16)])
def test_masks(dtype, P, mask):
    Case(dtype, 6, 2, 64, P, 203, 170, extra=37, mask=mask, seed=1).check()


@pytest.mark.parametrize("mask", ["causal", "random"])
@pytest.mark.parametrize("cap,bias,q_scale", [(15.0, False, 1.0), (0.0, True, 1.0), (2.0, True, 4.0), (30.0, True, 8.0),
                                              (1e4, False, 1.0), (1e-3, False, 1.0), (6.0, False, 1.0), (4.0, True, 1.0)])
@pytest.mark.parametrize("dtype,d,P", [("bf16", 128, 128), ("bf16", 64, 128), ("bf16", 64, 16), ("f32", 128, 32)])
def test_cap_and_bias(dtype, d, P, cap, bias, q_scale, mask):
    Case(dtype, 4, 2, d, P, 133, 140, extra=11, cap=cap, bias=bias, mask=mask, q_scale=q_scale, seed=3).check()


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("kw", [dict(cap=30.0), dict(cap=3.0), dict(bias=True), dict(cap=30.0, bias=True)])
def test_hidden_and_whole_halves_of_one_tile(kw, mask):
    """Ranges that end inside a page and inside its halves: tiles whose halves
    take different ways through the kernels share their rows' statistics."""
    Case("bf16", 4, 2, 128, 128, 530, 200, extra=100, mask=mask, seed=21, **kw).check()


@pytest.mark.parametrize("n", [1, 2, 5, 15, 16, 17, 63, 64, 65, 127, 128, 129, 257])
@pytest.mark.parametrize("dtype,Hq,Hkv,d,P,q_start", [
    ("bf16", 7, 1, 128, 128, 300), ("bf16", 8, 8, 64, 128, 0), ("f32", 6, 3, 64, 48, 61)])
def test_lengths(dtype, Hq, Hkv, d, P, q_start, n):
    Case(dtype, Hq, Hkv, d, P, q_start, n, cap=20.0, bias=n % 2 == 1, mask="window" if n % 3 else "causal", seed=n).check()


@pytest.mark.parametrize("Hq,Hkv,d,n,q_start", [(28, 4, 128, 1, 5000), (28, 4, 128, 4, 2047), (64, 8, 64, 1, 129),
                                                (16, 1, 64, 3, 4001), (32, 2, 128, 1, 1), (1, 1, 128, 1, 0)])
@pytest.mark.parametrize("mask", ["causal", "window"])
def test_single_tokens_against_long_caches(Hq, Hkv, d, n, q_start, mask):
    Case("bf16", Hq, Hkv, d, 128, q_start, n, cap=50.0, bias=True, mask=mask, seed=9).check()


@pytest.mark.parametrize("P", [16, 48, 64])
@pytest.mark.parametrize("Hq,Hkv,d,n,q_start,mask", [(28, 4, 128, 1, 1500, "causal"), (12, 4, 64, 9, 700, "random"),
                                                     (5, 1, 128, 16, 403, "docs"), (16, 8, 64, 7, 0, "future"),
                                                     (40, 2, 64, 2, 900, "pad"), (6, 6, 128, 3, 250, "empty")])
def test_few_queries_with_other_pages(P, Hq, Hkv, d, n, q_start, mask):
    """The few-query forward on pages smaller than a step of its keys (the backward on CUDA cores)."""
    Case("bf16", Hq, Hkv, d, P, q_start, n, extra=30, cap=40.0, bias=True, mask=mask, seed=10, q_scale=3.0).check()


@pytest.mark.parametrize("P", [8, 24])
def test_forward_with_small_pages(P):
    """Pages that are no multiple of 16 tokens: the forward takes them, the backward refuses."""
    for dtype in ("bf16", "f32"):
        c = Case(dtype, 4, 2, 64, P, 50, 33, cap=10.0, bias=True, mask="docs", seed=4)
        try:
            r, tol = c.oracle()
            o, lse = c.forward()
            B.pkv_check(c.pool)
            assert (np.abs(_f64(o) - r["o"]) <= tol["o"]).all() and (np.abs(_f64(lse) - r["lse"]) <= tol["lse"]).all()
            with pytest.raises(B.PkvError) as e:
                c.backward(o, lse)
            assert e.value.status == B.PKV_ERR_UNSUPPORTED
        finally:
            c.close()


@pytest.mark.parametrize("dtype,P,n,q_start,k", [("bf16", 128, 400, 1024, 3), ("bf16", 128, 130, 512, 9), ("f32", 16, 70, 96, 4)])
@pytest.mark.parametrize("mask", ["causal", "docs", "random"])
def test_page_selections(dtype, P, n, q_start, k, mask):
    """Selected pages and ranges together; pages outside every list get no gradient."""
    Case(dtype, 4, 2, 64, P, q_start, n, cap=5.0, bias=True, mask=mask, seed=6, sel=k).check()


def test_no_modification_is_the_plain_attention():
    """Neither cap nor bias nor ranges: the plain calls' results, to the bounds of both."""
    c = Case("bf16", 8, 2, 128, 128, 256, 200, seed=7)
    try:
        o, lse = c.forward()
        dq = c.backward(o, lse)
        dk, dv = c.grads()
        B.pkv_grad_zero(c.seq, torch.cuda.current_stream())
        o2, lse2, dq2 = torch.empty_like(o), torch.empty_like(lse), torch.empty_like(o)
        st = torch.cuda.current_stream()
        B.pkv_chunk_attn_fwd(c.seq, c.q, c.q_start, c.n, o2, lse2, None, st)
        B.pkv_chunk_attn_bwd(c.seq, c.q, o2, c.dout, lse2, c.q_start, c.n, dq2, None, st)
        dk2, dv2 = c.grads()
        B.pkv_check(c.pool)
        r, tol = c.oracle()
        # The plain LSE sums bf16-rounded weights: one more 2^-8 relative.
        for a, b, t in ((o, o2, tol["o"]), (dq, dq2, tol["dq"] * 2), (dk, dk2, tol["dk"] * 2), (dv, dv2, tol["dv"] * 2)):
            assert (np.abs(_f64(a) - _f64(b)) <= 2 * t).all()
        assert np.abs(_f64(lse) - _f64(lse2)).max() <= 2.0 ** -8 + tol["lse"].max()
    finally:
        c.close()


def test_gradients_accumulate_over_chunks_and_repeat():
    """Two chunks add into the same pages; a second sweep after zeroing repeats the first."""
    c = Case("bf16", 4, 2, 128, 128, 130, 260, cap=25.0, bias=True, mask="docs", seed=11)
    try:
        r, tol = c.oracle()
        st = torch.cuda.current_stream()
        cut = 101
        for _ in range(2):
            B.pkv_grad_zero(c.seq, st)
            for a, b in ((cut, 260), (0, cut)):
                mod = B.score_mod(c.cap, c.slopes.cuda(), c.k_begin[a:b].cuda(), c.k_end[a:b].cuda())
                o = torch.empty(b - a, 4, 128, dtype=c.dt, device="cuda")
                lse, dq = torch.empty(4, b - a, device="cuda"), torch.empty_like(o)
                B.pkv_chunk_attn_mod_fwd(c.seq, c.q[a:b], c.q_start + a, b - a, o, lse, mod, None, st)
                B.pkv_chunk_attn_mod_bwd(c.seq, c.q[a:b], o, c.dout[a:b], lse, c.q_start + a, b - a, dq, mod, None, st)
                assert (np.abs(_f64(dq) - r["dq"][a:b]) <= tol["dq"][a:b]).all()
            dk, dv = c.grads()
            B.pkv_check(c.pool)
            assert (np.abs(_f64(dk) - r["dk"]) <= tol["dk"]).all() and (np.abs(_f64(dv) - r["dv"]) <= tol["dv"]).all()
    finally:
        c.close()


def test_gradient_follows_differences():
    """fp32: <w, O> moved along a direction of q, and of the keys and values. The
    oracle's own central difference with the same step says what truncation
    leaves; the rest is rounding of O, within its bounds, over the step."""
    c = Case("f32", 4, 2, 64, 16, 40, 30, cap=3.0, bias=True, mask="docs", seed=13)
    try:
        r, tol = c.oracle()
        o, lse = c.forward()
        dq = c.backward(o, lse)
        dk, dv = c.grads()
        h, w = 2.0 ** -5, _f64(c.dout)
        g = torch.Generator().manual_seed(5)
        kept = {"q": c.q, "k": c.k, "v": c.v}
        for name, grad in (("q", dq), ("k", dk), ("v", dv)):
            step = torch.randn(kept[name].shape, generator=g).cuda()
            ours, exact, slack = [], [], 0.0
            for sign in (1, -1):
                x = dict(kept, **{name: kept[name] + sign * h * step})
                B.pkv_seq_reset(c.seq)
                B.pkv_append(c.seq, x["k"], x["v"], c.L, torch.cuda.current_stream())
                c.q = x["q"]
                ours.append((w * _f64(c.forward()[0])).sum())
                y = [_f64(x[t]) for t in "qkv"]
                rr = mod_oracle.attention(*y, c.q_start, **c.kw())
                exact.append((w * rr["o"]).sum())
                slack += (np.abs(w) * mod_oracle.bounds(rr, *y, c.q_start, False, **c.kw())["o"]).sum()
            c.q = kept["q"]
            diff = (ours[0] - ours[1]) / (2 * h)
            truncation = abs((exact[0] - exact[1]) / (2 * h) - (r["d" + name] * _f64(step)).sum())
            grad_err = (tol["d" + name] * np.abs(_f64(step))).sum()
            assert abs(diff - (_f64(grad) * _f64(step)).sum()) <= slack / (2 * h) + truncation + grad_err
    finally:
        c.close()


def test_rows_behind_the_chunk_and_its_outputs_are_left_alone():
    c = Case("bf16", 4, 1, 64, 128, 100, 77, extra=300, cap=9.0, mask="future", seed=14)
    try:
        st = torch.cuda.current_stream()
        o = torch.full((c.n + 8, c.Hq, c.d), 7.0, dtype=c.dt, device="cuda")
        lse = torch.full((c.Hq * c.n + 8,), 7.0, device="cuda")
        dq = torch.full_like(o, 7.0)
        B.pkv_chunk_attn_mod_fwd(c.seq, c.q, c.q_start, c.n, o[:c.n], lse[:c.Hq * c.n].view(c.Hq, c.n), c.mod, None, st)
        B.pkv_chunk_attn_mod_bwd(c.seq, c.q, o[:c.n], c.dout, lse[:c.Hq * c.n].view(c.Hq, c.n), c.q_start, c.n, dq[:c.n],
                                 c.mod, None, st)
        dk, dv = c.grads()
        B.pkv_check(c.pool)
        assert (o[c.n:] == 7).all() and (dq[c.n:] == 7).all() and (lse[c.Hq * c.n:] == 7).all()
        behind = c.q_start + c.n + 39                        # keys that no query's range reaches
        assert not dk[behind:].any() and not dv[behind:].any() and dk[:behind].any()
    finally:
        c.close()


def test_pinned_host_pool():
    """Staged pages; a window whose far pages are not staged and not touched."""
    n, d, P, Hq, Hkv, q_start = 128, 128, 128, 4, 2, 512
    c = Case("bf16", Hq, Hkv, d, P, q_start, n, cap=12.0, seed=15)
    pool = B.pkv_pool_create(P, Hkv, Hq, d, B.PKV_BF16, 5, residency=B.PKV_RES_PINNED_HOST, n_device_slots=2)
    try:
        seq = B.pkv_seq_create(pool)
        B.pkv_append(seq, c.k, c.v, c.L)
        lo = torch.full((n,), 400, dtype=torch.int64, device="cuda")
        c.k_begin, c.mod = lo.cpu(), B.score_mod(c.cap, None, lo)
        pages = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
        B.pkv_prefetch(seq, pages, 2, 3)
        B.pkv_wait(seq)
        o, lse = torch.empty(n, Hq, d, dtype=c.dt, device="cuda"), torch.empty(Hq, n, device="cuda")
        dq = torch.empty_like(o)
        B.pkv_chunk_attn_mod_fwd(seq, c.q, q_start, n, o, lse, c.mod)
        B.pkv_chunk_attn_mod_bwd(seq, c.q, o, c.dout, lse, q_start, n, dq, c.mod)
        B.pkv_writeback_grads(seq)
        dk, dv = (torch.empty(c.L, Hkv, d, device="cuda") for _ in range(2))
        B.pkv_gather(seq, dk=dk, dv=dv)
        B.pkv_check(pool)
        r, tol = c.oracle()
        for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
            assert (np.abs(_f64(t) - r[name]) <= tol[name]).all(), name
    finally:
        B.pkv_pool_destroy(pool)
        c.close()


@pytest.mark.parametrize("n,q_start", [(1, 3000), (140, 260)])
def test_captured_graph_on_a_side_stream(n, q_start):
    """Forward and backward replayed from a graph while the scratch has grown
    since, with new queries; a capture that would need more scratch refuses."""
    c = Case("bf16", 8, 2, 64, 128, q_start, n, cap=30.0, mask="window", seed=16)
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o, lse, dq = torch.empty_like(c.q), torch.empty(c.Hq, n, device="cuda"), torch.empty_like(c.q)
        torch.cuda.synchronize()

        def both(stream):
            B.pkv_chunk_attn_mod_fwd(c.seq, c.q, q_start, n, o, lse, c.mod, None, stream)
            B.pkv_grad_zero(c.seq, stream)
            B.pkv_chunk_attn_mod_bwd(c.seq, c.q, o, c.dout, lse, q_start, n, dq, c.mod, None, stream)

        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            with pytest.raises(B.PkvError) as e:
                both(side)
                B.pkv_chunk_attn_mod_bwd(c.seq, c.q, o, c.dout, lse, q_start, n, dq, c.mod, None, side)
            assert "before capturing" in str(e.value)
        both(side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(side)
        # A longer call grows the scratch: the graph's buffer has to live on.
        big = min(400, c.L)
        q2 = torch.randn(big, c.Hq, c.d, device="cuda").to(c.dt)
        o2, lse2 = torch.empty_like(q2), torch.empty(c.Hq, big, device="cuda")
        m2 = B.score_mod(c.cap)
        B.pkv_chunk_attn_mod_fwd(c.seq, q2, 0, big, o2, lse2, m2)
        B.pkv_chunk_attn_mod_bwd(c.seq, q2, o2, q2, lse2, 0, big, torch.empty_like(q2), m2)
        torch.cuda.synchronize()
        for seed in (1, 2):
            c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator().manual_seed(seed)))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            dk, dv = c.grads()
            B.pkv_check(c.pool)
            r, tol = c.oracle()
            for name, t in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
                assert (np.abs(_f64(t) - r[name]) <= tol[name]).all(), name
    finally:
        c.close()


def test_repeated_calls_are_bit_identical():
    for n, q_start in ((300, 900), (1, 4000), (3, 700)):
        c = Case("bf16", 28, 4, 128, 128, q_start, n, cap=50.0, bias=True, mask="docs", seed=17)
        try:
            first = c.forward()
            dq = c.backward(*first)
            for _ in range(20):
                again = c.forward()
                assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
                assert torch.equal(dq, c.backward(*again))
        finally:
            c.close()


def test_empty_chunk():
    c = Case("bf16", 4, 2, 64, 128, 40, 10, seed=18)
    try:
        e = torch.empty(0, 4, 64, dtype=c.dt, device="cuda")
        lse = torch.empty(4, 0, device="cuda")
        m = B.score_mod(5.0)
        B.pkv_chunk_attn_mod_fwd(c.seq, e, 50, 0, e, lse, m)
        B.pkv_chunk_attn_mod_bwd(c.seq, e, e, e, lse, 50, 0, e, m)
        B.pkv_check(c.pool)
    finally:
        c.close()
