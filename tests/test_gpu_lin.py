"""Linear attention with a decay per head against its recurrence in float64.

Bounds, from the arithmetic. Every output is a sum of products; mag is the same
sum over absolute values. float32 work: at most d additions in a product over the
head dimension, 128 over a chunk, one per chunk in the scan, and a few factors: at
most (d + 128 + chunks + 16) 2^-24 mag; a decay l^m = 2^(m log2 l) is off by
m |log2 l| 2^-23 relative, below 40 * 2^-23 for all weights down to 2^-40 (smaller
ones are within that of nothing). So F = (d + 224 + chunks) 2^-24 covers both.
bf16 products on the tensor cores round one factor of each term to bf16 (a
chunk's weighted scores, or the state a chunk starts from or its gradient): 2^-8
mag more (half a step); states and their gradients carry no such rounding. Storage
rounds an output once: half an eps of its type.
"""
import numpy as np
import pytest
import torch

import lin_oracle as O
from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu

DT = {"bf16": (torch.bfloat16, B.PKV_BF16), "f32": (torch.float32, B.PKV_F32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


class Memory:
    def __init__(self, address, shape):
        self.__cuda_array_interface__ = {"shape": shape, "typestr": "<f4", "data": (address, False), "version": 2}


class Store:
    def __init__(self, dtype, Hq, Hkv, d, slots, grads=True, flags=0):
        self.lin = B.pkv_lin_create(Hkv, Hq, d, DT[dtype][1], slots, grads=grads, flags=flags)
        at = B.pkv_lin_arrays(self.lin)
        self.state, self.dstate = (torch.as_tensor(Memory(at[x], (slots, Hkv, d, d)), device="cuda") if at[x] else None
                                   for x in ("state", "dstate"))

    def __enter__(self):
        return self

    def __exit__(self, *_):
        torch.cuda.synchronize()
        B.pkv_lin_destroy(self.lin)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _decays(kind, Hkv):
    if kind is None:
        return None
    return torch.tensor({"spread": np.linspace(-0.3, -0.002, Hkv), "zero": np.zeros(Hkv), "fast": np.linspace(-6.0, -1.0, Hkv),
                         "own": np.full(Hkv, -np.inf)}[kind], dtype=torch.float32)


def _rows(n, heads, d, dt, strided, seed):
    """Tensors [n, h, d]: slices of one tensor with a gap behind each row, or dense."""
    g = torch.Generator().manual_seed(seed)
    if strided:
        return torch.randn(n, sum(heads) + 1, d, generator=g).to(dt).cuda()[:, :sum(heads)].split(heads, dim=1)
    return tuple(torch.randn(n, h, d, generator=g).to(dt).cuda() for h in heads)


def _close(got, want, mag, c, dt, what):
    want, mag = np.asarray(want), np.asarray(mag)
    half = torch.finfo(dt).eps / 2
    tol = c * mag + half * (np.abs(want) + c * mag)
    over = np.abs(_f64(got) - want) - tol
    assert not np.isnan(over).any() and over.max(initial=0) <= 0, (what, over.max(), np.argmax(over))


CASES = [
    # dtype, Hq, Hkv, d, cuts (rows before the first and behind the last are no sequence's), decay, first state, strided
    ("bf16", 4, 2, 128, [0, 1], "spread", True, False),
    ("bf16", 7, 1, 128, [0, 300], "spread", True, True),
    ("bf16", 4, 4, 64, [0, 128], None, False, False),
    ("bf16", 4, 2, 64, [0, 127, 128, 128, 385], "spread", True, True),
    ("bf16", 6, 2, 128, [3, 67, 196, 196, 325, 330], "fast", True, False),
    ("bf16", 2, 1, 128, [0, 640], "zero", True, False),
    ("bf16", 3, 3, 64, [5, 134], "own", True, True),
    ("bf16", 20, 1, 64, [0, 0, 65], "spread", False, False),
    ("f32", 2, 1, 64, [0, 1], "fast", True, True),
    ("f32", 4, 2, 64, [0, 63, 64, 64, 201], "spread", True, False),
    ("f32", 3, 1, 128, [7, 71, 200], "zero", True, True),
    ("f32", 4, 4, 128, [0, 65], "own", False, False),
]


def _oracle(x, cuts, decay, first, dlast, fn=lambda t: t):
    """All sequences by the recurrence: per output a full array (zero where no sequence is); fn: abs for the bounds."""
    q, k, v, do = (fn(_f64(t)) for t in x)
    out = {"o": np.zeros(q.shape), "dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(k.shape), "state": [], "dstate": []}
    for b, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        s = slice(lo, hi)
        out["o"][s], last = O.lin_forward(q[s], k[s], v[s], decay, fn(first[b]))
        out["dq"][s], out["dk"][s], out["dv"][s], g = O.lin_backward(q[s], k[s], v[s], do[s], decay, fn(first[b]), fn(dlast[b]))
        out["state"].append(last)
        out["dstate"].append(g)
    return out


@pytest.mark.parametrize("flags", [0, B.PKV_FLAG_SIMT_ONLY])
@pytest.mark.parametrize("dtype,Hq,Hkv,d,cuts,kind,start,strided", CASES)
def test_forward_and_backward(dtype, Hq, Hkv, d, cuts, kind, start, strided, flags):
    if dtype == "f32" and flags:
        pytest.skip("the same kernels")
    dt, m, n = DT[dtype][0], len(cuts) - 1, cuts[-1] + 9
    q, k, v, do = _rows(n, (Hq, Hkv, Hkv, Hq), d, dt, strided, n)
    outside = torch.ones(n, dtype=torch.bool)
    outside[cuts[0]:cuts[-1]] = False
    for t in (q, k, v, do):
        t[outside] = float("nan")                     # rows of no sequence are not read
    log_decay = _decays(kind, Hkv)
    decay = np.ones(Hkv) if log_decay is None else np.exp(log_decay.double().numpy())
    r = np.random.default_rng(n)
    first, dlast = (r.standard_normal((m, Hkv, d, d)).astype(np.float32).astype(float) for _ in range(2))
    if not start:
        first[:] = 0
    with Store(dtype, Hq, Hkv, d, 2 * m + 1, flags=flags) as c:
        c.state.fill_(7.0)
        c.dstate.fill_(5.0)
        order = torch.randperm(2 * m + 1, generator=torch.Generator().manual_seed(n)).to(torch.int32).cuda()
        src, dst = order[:m].contiguous(), order[m:2 * m].contiguous()
        if start:
            c.state[src.long()] = torch.tensor(first, dtype=torch.float32, device="cuda")
        c.dstate[dst.long()] = torch.tensor(dlast, dtype=torch.float32, device="cuda")
        cu = torch.tensor(cuts, device="cuda")
        batch = B.lin_batch(m, cu, src if start else None, dst)
        o, dq, dk, dv = (torch.full((n, h, d), 3.0, dtype=dt, device="cuda") for h in (Hq, Hq, Hkv, Hkv))
        g2 = None if log_decay is None else log_decay.cuda()
        st = torch.cuda.current_stream()
        B.pkv_lin_attn_fwd(c.lin, q, k, v, o, n, g2, batch, st)
        B.pkv_lin_attn_bwd(c.lin, q, k, v, do, dq, dk, dv, n, g2, batch, st)
        B.pkv_lin_check(c.lin)
        x = [torch.nan_to_num(t) for t in (q, k, v, do)]
        want, mag = _oracle(x, cuts, decay, first, dlast), _oracle(x, cuts, decay, first, dlast, np.abs)
        F = (d + 224 + n // 64) * 2.0 ** -24
        W = F if dtype == "f32" or flags else F + 2.0 ** -8
        inside = ~outside.numpy()
        for name, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
            _close(t[~outside], want[name][inside], mag[name][inside], W, dt, name)
            assert (t[outside] == 3.0).all()           # left as they were
        _close(c.state[dst.long()], want["state"], mag["state"], F, torch.float32, "state")
        if start:
            _close(c.dstate[src.long()], want["dstate"], mag["dstate"], F, torch.float32, "dstate")
        else:
            assert (c.state[src.long()] == 7.0).all()
        rest = order[2 * m:].long()
        assert (c.state[rest] == 7.0).all() and (c.dstate[rest] == 5.0).all()


@pytest.mark.parametrize("dtype,Hq,Hkv,d,n", [("bf16", 28, 4, 128, 5), ("bf16", 3, 3, 64, 1), ("bf16", 40, 2, 64, 3),
                                              ("f32", 4, 2, 64, 17), ("f32", 17, 1, 128, 2)])
@pytest.mark.parametrize("kind", ["spread", None, "own"])
def test_step(dtype, Hq, Hkv, d, n, kind):
    """Three tokens for each of the batch's live rows, slots in no order, padding rows between."""
    dt = DT[dtype][0]
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    if n > 1:
        slots[n // 2] = -1
    log_decay = _decays(kind, Hkv)
    decay = np.ones(Hkv) if log_decay is None else np.exp(log_decay.double().numpy())
    with Store(dtype, Hq, Hkv, d, n + 2, grads=False) as c:
        c.state.copy_(torch.randn(c.state.shape, generator=torch.Generator().manual_seed(1)))
        S = _f64(c.state)
        M = np.abs(S)
        for t in range(3):
            q, k, v = _rows(n, (Hq, Hkv, Hkv), d, dt, t == 1, 10 * n + t)
            o = torch.full((n, Hq, d), 3.0, dtype=dt, device="cuda")
            B.pkv_lin_attn_step(c.lin, q, k, v, o, n, None if log_decay is None else log_decay.cuda(), slots.cuda(),
                                torch.cuda.current_stream())
            F = (d + 24 + 3 * t) * 2.0 ** -24
            for i, s in enumerate(slots.tolist()):
                if s < 0:
                    assert (o[i] == 3.0).all()
                    continue
                one = [_f64(x[i:i + 1]) for x in (q, k, v)]
                want, S[s] = O.lin_forward(*one, decay, S[s])
                mag, M[s] = O.lin_forward(*map(np.abs, one), decay, M[s])
                _close(o[i:i + 1], want, mag, F, dt, ("o", t, i))
            _close(c.state, S, M, F, torch.float32, ("state", t))
        B.pkv_lin_check(c.lin)


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [("bf16", 14, 2, 64), ("f32", 2, 1, 128)])
def test_prompt_in_pieces_then_steps(dtype, Hq, Hkv, d):
    """A prompt by forward calls of several lengths in place on one slot, the rest by steps: the
    recurrence over the whole; and the backward of the pieces in reverse, states in slots of their own."""
    dt, cuts = DT[dtype][0], [0, 130, 131, 200, 456]
    n = cuts[-1] + 3
    q, k, v, do = _rows(n, (Hq, Hkv, Hkv, Hq), d, dt, True, 5)
    log_decay = _decays("spread", Hkv)
    decay = np.exp(log_decay.double().numpy())
    g2, st = log_decay.cuda(), torch.cuda.current_stream()
    zero = np.zeros((1, Hkv, d, d))
    want, mag = (_oracle((q, k, v, do), [0, n], decay, zero, zero, f) for f in (lambda t: t, np.abs))
    cut = cuts[-1]
    part, pmag = (_oracle([t[:cut] for t in (q, k, v, do)], [0, cut], decay, zero, zero, f) for f in (lambda t: t, np.abs))
    F = (d + 224 + n // 64) * 2.0 ** -24
    W = F + (2.0 ** -8 if dtype == "bf16" else 0)
    with Store(dtype, Hq, Hkv, d, 6) as c:
        o = torch.empty(n, Hq, d, dtype=dt, device="cuda")
        same = torch.tensor([5], dtype=torch.int32, device="cuda")
        for lo, hi in zip(cuts, cuts[1:]):             # c.state[5] starts at zero
            B.pkv_lin_attn_fwd(c.lin, q[lo:hi], k[lo:hi], v[lo:hi], o[lo:hi], hi - lo, g2, B.lin_batch(1, None, same, same), st)
        for t in range(cut, n):
            B.pkv_lin_attn_step(c.lin, q[t:t + 1], k[t:t + 1], v[t:t + 1], o[t:t + 1], 1, g2, same, st)
        _close(o, want["o"], mag["o"], W, dt, "o")
        _close(c.state[5:], want["state"], mag["state"], F, torch.float32, "state")
        at = torch.arange(6, dtype=torch.int32, device="cuda")
        dq, dk, dv = (torch.empty(n, h, d, dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
        for i, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
            batch = B.lin_batch(1, None, at[i:i + 1] if i else None, at[i + 1:i + 2])
            B.pkv_lin_attn_fwd(c.lin, q[lo:hi], k[lo:hi], v[lo:hi], o[lo:hi], hi - lo, g2, batch, st)
        for i in reversed(range(len(cuts) - 1)):
            lo, hi = cuts[i:i + 2]
            batch = B.lin_batch(1, None, at[i:i + 1] if i else None, at[i + 1:i + 2] if i + 2 < len(cuts) else None)
            B.pkv_lin_attn_bwd(c.lin, *(t[lo:hi] for t in (q, k, v, do, dq, dk, dv)), hi - lo, g2, batch, st)
        B.pkv_lin_check(c.lin)
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            _close(t[:cut], part[name], pmag[name], W, dt, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows_hand_the_state_on(dtype):
    with Store(dtype, 2, 1, 64, 4) as c:
        c.state.copy_(torch.randn(c.state.shape))
        c.dstate.copy_(torch.randn(c.state.shape))
        keep, dkeep = c.state.clone(), c.dstate.clone()
        i = torch.arange(4, dtype=torch.int32, device="cuda")
        e = torch.empty(0, 2, 64, dtype=DT[dtype][0], device="cuda")
        f = e[:, :1].contiguous()
        for batch in (B.lin_batch(1, None, i[:1], i[2:3]), B.lin_batch(2, torch.zeros(3, dtype=torch.int64, device="cuda"), i[:2], i[2:])):
            B.pkv_lin_attn_fwd(c.lin, e, f, f, e, 0, None, batch)
            B.pkv_lin_attn_bwd(c.lin, e, f, f, e, e, f, f, 0, None, batch)
        B.pkv_lin_attn_step(c.lin, e, f, f, e, 0, None, i[:0])
        B.pkv_lin_attn_fwd(c.lin, e, f, f, e, 0, None, B.lin_batch(0, torch.zeros(1, dtype=torch.int64, device="cuda")))
        B.pkv_lin_check(c.lin)
        assert torch.equal(c.state, torch.cat([keep[:2], keep[:2]])) and torch.equal(c.dstate, torch.cat([dkeep[2:], dkeep[2:]]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_ranges_and_slots_are_recorded(dtype):
    """Checked by the kernels before any access: the sequence is left out, the store stays usable."""
    dt = DT[dtype][0]
    n = 150
    q, k, v, do = _rows(n, (2, 1, 1, 2), 64, dt, False, 1)
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    with Store(dtype, 2, 1, 64, 2) as c:
        def fwd(cu=None, a=None, b=None):
            o = torch.full_like(q, 3.0)
            B.pkv_lin_attn_fwd(c.lin, q, k, v, o, n, None, B.lin_batch(1 if cu is None else len(cu) - 1, None if cu is None else
                                                                      torch.tensor(cu, device="cuda"), a, b))
            return o
        for cu in ([0, n + 1], [-1, 5], [9, 4], [0, 1 << 40], [-(1 << 40), -5], [1 << 62, 1 << 62]):
            o = fwd(cu)
            with pytest.raises(B.PkvError, match="range"):
                B.pkv_lin_check(c.lin)
            assert (o == 3.0).all()
            g = [torch.full_like(t, 3.0) for t in (q, k, v)]
            B.pkv_lin_attn_bwd(c.lin, q, k, v, do, *g, n, None, B.lin_batch(1, torch.tensor(cu, device="cuda")))
            with pytest.raises(B.PkvError, match="range"):
                B.pkv_lin_check(c.lin)
            assert all((t == 3.0).all() for t in g)
        for bad in (2, -2, 2 ** 31 - 1):
            for a, b in ((i + bad, None), (None, i + bad)):
                fwd(None, a, b)
                with pytest.raises(B.PkvError, match="slot"):
                    B.pkv_lin_check(c.lin)
            o = torch.full_like(q[:1], 3.0)
            B.pkv_lin_attn_step(c.lin, q[:1], k[:1], v[:1], o, 1, None, i + bad)
            with pytest.raises(B.PkvError, match="slot"):
                B.pkv_lin_check(c.lin)
            assert (o == 3.0).all()
        assert not c.state.any()
        good = fwd(None, None, i)                      # usable as before
        B.pkv_lin_check(c.lin)
        assert torch.equal(good, fwd([0, n]))


@pytest.mark.parametrize("dtype,flags,Hkv", [("bf16", 0, 1), ("bf16", B.PKV_FLAG_SIMT_ONLY, 2), ("f32", 0, 2)])
def test_a_slot_given_twice_is_recorded(dtype, flags, Hkv):
    """Two sequences of one call on one slot: recorded (every access stays inside the store);
    what is allowed, a slot read for several or read and written for one, is not."""
    dt = DT[dtype][0]
    n, m = 300, 200
    q, k, v, do = _rows(n, (2 * Hkv, Hkv, Hkv, 2 * Hkv), 64, dt, False, 1)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = torch.arange(m + 1, device="cuda")
    ids = list(range(m))
    last = ids[:-1] + [3]                        # the last sequence's is the fourth's
    other = [-1] * (m - 1) + [7]                 # the last starts from what the eighth writes
    with Store(dtype, 2 * Hkv, Hkv, 64, m, flags=flags) as c:
        def check(bad):
            if not bad:
                return B.pkv_lin_check(c.lin)
            with pytest.raises(B.PkvError, match="two sequences"):
                B.pkv_lin_check(c.lin)
        for start, end, bad in ((None, ids, False), (ids, ids, False), ([5] * m, None, False), (None, last, True), (other, ids, True),
                                (other, [-1] * m, False)):
            start, end = (None if x is None else dev(x) for x in (start, end))
            B.pkv_lin_attn_fwd(c.lin, q, k, v, torch.empty_like(q), n, None, B.lin_batch(m, cu, start, end))
            check(bad)
        for start, end, bad in ((ids, ids, False), (ids, None, False), (last, None, True), ([5] * m, None, True), (ids, other, True)):
            start, end = (None if x is None else dev(x) for x in (start, end))
            g = [torch.empty_like(t) for t in (q, k, v)]
            B.pkv_lin_attn_bwd(c.lin, q, k, v, do, *g, n, None, B.lin_batch(m, cu, start, end))
            check(bad)
        for slots, bad in ((ids, False), (last, True), ([-1] * m, False), ([0, -1] + [9] * (m - 2), True)):
            B.pkv_lin_attn_step(c.lin, q[:m], k[:m], v[:m], torch.empty_like(q[:m]), m, None, dev(slots))
            check(bad)


@pytest.mark.parametrize("Hq,Hkv,d,n,dtype", [(16, 16, 128, 10000, "bf16"), (32, 16, 64, 11111, "bf16"), (3, 1, 64, 5000, "f32")])
def test_a_long_call_equals_its_pieces(Hq, Hkv, d, n, dtype):
    """Pieces of whole chunks, their states handed on through slots: the same sums in the same
    order, so the same bits, however the work is laid out over the GPU."""
    q, k, v, do = _rows(n, (Hq, Hkv, Hkv, Hq), d, DT[dtype][0], False, 5)
    cuts = [0, 1280, 1408, 4096, n]
    g2 = _decays("spread", Hkv).cuda()
    i = torch.arange(len(cuts), dtype=torch.int32, device="cuda")
    got = []
    for ends in ([0, n], cuts):
        with Store(dtype, Hq, Hkv, d, len(cuts)) as c:
            gen = torch.Generator(device="cuda").manual_seed(9)
            c.state[0] = torch.randn(Hkv, d, d, device="cuda", generator=gen)
            c.dstate[len(ends) - 1] = torch.randn(Hkv, d, d, device="cuda", generator=gen)
            o, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
            spans = list(enumerate(zip(ends, ends[1:])))
            batch = lambda x: B.lin_batch(1, None, i[x:x + 1], i[x + 1:x + 2])  # noqa: E731
            for x, (a, b) in spans:
                B.pkv_lin_attn_fwd(c.lin, q[a:b], k[a:b], v[a:b], o[a:b], b - a, g2, batch(x))
            for x, (a, b) in reversed(spans):
                B.pkv_lin_attn_bwd(c.lin, q[a:b], k[a:b], v[a:b], do[a:b], dq[a:b], dk[a:b], dv[a:b], b - a, g2, batch(x))
            B.pkv_lin_check(c.lin)
            got.append([o, dq, dk, dv, c.state[len(ends) - 1].clone(), c.dstate[0].clone()])
    for name, a, b in zip(("o", "dq", "dk", "dv", "state", "dstate"), *got):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dtype,m", [("bf16", 33), ("bf16", 1025), ("f32", 1100), ("bf16", 9000)])
def test_many_sequences_equal_each_by_itself(dtype, m):
    """More sequences than a warp has lanes, or than its square: the bits of calls of 30 at a time
    (every chunk of every sequence is found), both ways; 9000 by a sample of those."""
    g = torch.Generator().manual_seed(m)
    lens = torch.randint(0, 5, (m,), generator=g)
    lens[torch.randint(0, m, (3,), generator=g)] = 300
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]) + 2
    n = int(cu[-1]) + 3
    Hq, Hkv, d = 2, 1, 64
    q, k, v, do = _rows(n, (Hq, Hkv, Hkv, Hq), d, DT[dtype][0], False, 6)
    g2 = _decays("spread", Hkv).cuda()
    ids = torch.arange(m, dtype=torch.int32, device="cuda")
    starts = list(range(0, m, 30)) if m < 2000 else [0, 1020, 4980, 8970]
    with Store(dtype, Hq, Hkv, d, m) as c:
        first = torch.randn(m, Hkv, d, d, device="cuda")
        got = []
        for calls in ([(0, m)], [(b, min(m, b + 30)) for b in starts]):
            c.state.copy_(first)
            c.dstate.copy_(first)
            o, dq, dk, dv = (torch.full_like(t, 3.0) for t in (q, q, k, v))
            for a, b in calls:
                batch = B.lin_batch(b - a, cu[a:b + 1].cuda(), ids[a:b], ids[a:b])
                B.pkv_lin_attn_bwd(c.lin, q, k, v, do, dq, dk, dv, n, g2, batch)
                B.pkv_lin_attn_fwd(c.lin, q, k, v, o, n, g2, batch)
            B.pkv_lin_check(c.lin)
            got.append([o, dq, dk, dv, c.state.clone(), c.dstate.clone()])
        for x, (a, b) in enumerate(zip(*got)):
            for s in starts:
                e = min(m, s + 30)
                at = slice(s, e) if x >= 4 else slice(int(cu[s]), int(cu[e]))
                assert torch.equal(a[at], b[at]), (x, s)
            assert x >= 4 or ((a[:2] == 3.0).all() and (a[int(cu[-1]):] == 3.0).all())


@pytest.mark.parametrize("dtype,flags", [("bf16", 0), ("bf16", B.PKV_FLAG_SIMT_ONLY), ("f32", 0)])
def test_graphs_streams_and_repeats(dtype, flags):
    """The same bits on another stream, from a captured graph replayed on new inputs, and again."""
    dt, n, Hq, Hkv, d = DT[dtype][0], 700, 6, 2, 64
    cu, m = torch.tensor([0, 300, 301, 690], device="cuda"), 3
    g2 = _decays("spread", Hkv).cuda()
    i = torch.arange(2 * m, dtype=torch.int32, device="cuda")
    sets = [_rows(n, (Hq, Hkv, Hkv, Hq), d, dt, False, s) for s in (1, 2)]
    with Store(dtype, Hq, Hkv, d, 2 * m, flags=flags) as c:
        c.state[:m] = torch.randn(m, Hkv, d, d, device="cuda")
        c.dstate[m:] = torch.randn(m, Hkv, d, d, device="cuda")
        x = [t.clone() for t in sets[0]]
        outs = [torch.zeros(n, h, d, dtype=dt, device="cuda") for h in (Hq, Hq, Hkv, Hkv)]

        def both(stream):
            batch = B.lin_batch(m, cu, i[:m], i[m:])
            B.pkv_lin_attn_fwd(c.lin, *x[:3], outs[0], n, g2, batch, stream)
            B.pkv_lin_attn_bwd(c.lin, *x, *outs[1:], n, g2, batch, stream)
            return batch

        def result():
            torch.cuda.synchronize()
            return [t.clone() for t in outs] + [c.state[m:].clone(), c.dstate[:m].clone()]

        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):     # no call has been made: nothing is allocated under a capture
            with pytest.raises(B.PkvError, match="once before capturing"):
                both(side)
        want = []
        for s in sets:
            for t, u in zip(x, s):
                t.copy_(u)
            both(torch.cuda.current_stream())
            want.append(result())
        side.wait_stream(torch.cuda.current_stream())
        both(side)
        assert all(torch.equal(a, b) for a, b in zip(result(), want[1]))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            keep = both(side)
        for s, w in zip(sets, want):
            for t, u in zip(x, s):
                t.copy_(u)
            for t in outs:
                t.zero_()
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(result(), w))
        del keep
        B.pkv_lin_check(c.lin)


def test_several_sequences_may_start_from_one_state():
    """A shared prefix: one state read for three sequences, and -1 for the fourth."""
    dt, Hq, Hkv, d, n = torch.bfloat16, 4, 2, 64, 260
    q, k, v, _ = _rows(n, (Hq, Hkv, Hkv, Hq), d, dt, False, 3)
    cuts = [0, 5, 140, 200, n]
    with Store("bf16", Hq, Hkv, d, 5) as c:
        c.state[0] = torch.randn(Hkv, d, d, device="cuda")
        one = [torch.empty(n, Hq, d, dtype=dt, device="cuda") for _ in range(2)]
        src = torch.tensor([0, 0, 0, -1], dtype=torch.int32, device="cuda")
        dst = torch.arange(1, 5, dtype=torch.int32, device="cuda")
        B.pkv_lin_attn_fwd(c.lin, q, k, v, one[0], n, None, B.lin_batch(4, torch.tensor(cuts, device="cuda"), src, dst))
        last = c.state[1:].clone()
        for b, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
            B.pkv_lin_attn_fwd(c.lin, q[lo:hi], k[lo:hi], v[lo:hi], one[1][lo:hi], hi - lo, None,
                               B.lin_batch(1, None, src[b:b + 1], dst[b:b + 1]))
        B.pkv_lin_check(c.lin)
        assert torch.equal(*one) and torch.equal(last, c.state[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_at_once_and_outgrown_scratch(dtype):
    """Two stores on two streams, steps on different slots of one store on two streams, and a graph
    that was captured before its store's scratch was outgrown: the bits of each by itself."""
    dt, Hq, Hkv, d, n = DT[dtype][0], 4, 2, 128, 900
    g2 = _decays("spread", Hkv).cuda()
    sets = [_rows(n, (Hq, Hkv, Hkv, Hq), d, dt, False, s) for s in (1, 2)]
    i = torch.arange(2, dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    with Store(dtype, Hq, Hkv, d, 2) as a, Store(dtype, Hq, Hkv, d, 2) as b:
        batch = B.lin_batch(1, None, i[:1], i[1:])

        def run(c, x, o, grads, stream, m=n):
            B.pkv_lin_attn_fwd(c.lin, *(t[:m] for t in x[:3]), o[:m], m, g2, batch, stream)
            B.pkv_lin_attn_bwd(c.lin, *(t[:m] for t in x), *(t[:m] for t in grads), m, g2, batch, stream)

        def fresh():
            return [torch.zeros_like(sets[0][0])] + [torch.zeros_like(t) for t in sets[0][:3]]
        want = []
        for x in sets:
            out = fresh()
            run(a, x, out[0], out[1:], torch.cuda.current_stream())
            torch.cuda.synchronize()
            want.append(out)
        for _ in range(3):
            outs = [fresh(), fresh()]
            torch.cuda.synchronize()
            for c, x, out, stream in zip((a, b), sets, outs, streams):
                run(c, x, out[0], out[1:], stream)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for out, w in zip(outs, want) for p, q in zip(out, w))
        # A graph of a short call, then a longer call that needs more scratch, then the graph again.
        with Store(dtype, Hq, Hkv, d, 2) as c:
            out, short = fresh(), fresh()
            run(c, sets[0], short[0], short[1:], torch.cuda.current_stream(), 300)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=streams[0]):
                run(c, sets[0], out[0], out[1:], streams[0], 300)
            long = fresh()
            run(c, sets[1], long[0], long[1:], torch.cuda.current_stream())
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, short)) and all(torch.equal(p, q) for p, q in zip(long, want[1]))
            B.pkv_lin_check(c.lin)
        # Single tokens: slot 0 on one stream, slot 1 on the other, five tokens each.
        states = []
        for at_once in (False, True):
            for c in (a, b):
                c.state.fill_(0.5)
            torch.cuda.synchronize()
            os = [torch.zeros(5, Hq, d, dtype=dt, device="cuda") for _ in range(2)]
            torch.cuda.synchronize()
            for s in range(2):
                for t in range(5):
                    q, k, v = (z[t:t + 1] for z in sets[s][:3])
                    B.pkv_lin_attn_step(a.lin, q, k, v, os[s][t:t + 1], 1, g2, i[s:s + 1], streams[s])
                if not at_once:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            states.append([a.state.clone(), *os])
        assert all(torch.equal(p, q) for p, q in zip(*states))
        B.pkv_lin_check(a.lin)
        B.pkv_lin_check(b.lin)
