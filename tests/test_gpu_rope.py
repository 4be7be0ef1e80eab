"""The rotated append, the rotation alone and their gradient, against the
definition in 64 bits or more.

Bounds, from the arithmetic. A turned element is a c - b s. The phase is
rounded to 2^-25 half turns (pi 2^-25 = 9.4e-8), sincospif is within 2 ulp
(1.2e-7 at 1), each product and the sum round by 2^-24 (6e-8, the sum's
relative to at most |a| + |b|): in all below 4e-7 (|a| + |b|); 2^-21 is used.
Storage then rounds once: half an eps of the type, relative. The angle itself
is exact modulo one turn; the oracle forms it in long double (64 or 113 bits).
"""
import math

import numpy as np
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu

ROT = 2.0 ** -21
DT = {"bf16": (torch.bfloat16, B.PKV_BF16), "f32": (torch.float32, B.PKV_F32)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inv_freq(rotary, theta=1e6):
    return torch.tensor([theta ** (-2.0 * i / rotary) for i in range(rotary // 2)], dtype=torch.float32)


def _turn(x, inv_freq, pos, interleaved, sign=1):
    """x [n, H, d] float64 turned; also the bound's |a| + |b| per element."""
    f = inv_freq.numpy().astype(np.longdouble)
    ang = sign * np.asarray(pos).astype(np.longdouble)[:, None, None] * f
    c, s = np.cos(ang).astype(np.float64), np.sin(ang).astype(np.float64)
    half = len(f)
    i = np.arange(half) * 2 if interleaved else np.arange(half)
    j = i + 1 if interleaved else i + half
    y, mag = x.copy(), np.zeros_like(x)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    mag[..., i] = mag[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return y, mag


def _close(got, want, mag, dt):
    tol = ROT * mag + (torch.finfo(dt).eps / 2) * (np.abs(want) + ROT * mag)
    bad = np.abs(_f64(got) - want) - tol
    assert bad.max() <= 0, (bad.max(), np.argmax(bad))


def _rows(n, heads, d, dt, fused, seed):
    """Q, K, V [n, h, d]: slices of one tensor with a gap behind each row, or dense."""
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn(n, sum(heads) + 1, d, generator=g).to(dt).cuda()
        return x[:, :sum(heads)].split(heads, dim=1)
    return tuple(torch.randn(n, h, d, generator=g).to(dt).cuda() for h in heads)


def _reps(k_rows, P):
    n = len(k_rows)
    return np.stack([k_rows[p:min(n, p + P)].mean(0) for p in range(0, n, P)])


CASES = [
    # dtype, Hq, Hkv, d, P, n, rotary, interleaved, fused, pos0
    ("bf16", 28, 4, 128, 128, 1, 128, False, False, 20011),
    ("bf16", 28, 4, 128, 128, 300, 128, False, True, 0),
    ("bf16", 7, 1, 128, 128, 129, 64, True, True, 5),
    ("bf16", 6, 2, 64, 16, 77, 64, False, False, 1000003),
    ("bf16", 5, 5, 64, 8, 31, 16, True, False, -40),
    ("bf16", 3, 1, 128, 24, 50, 48, False, True, 7),
    ("f32", 2, 1, 64, 16, 201, 32, True, False, 0),
    ("f32", 4, 2, 128, 64, 65, 128, False, True, 2 ** 31 - 70),
    ("f32", 9, 3, 64, 8, 8, 64, False, False, 123456789),
    ("f32", 4, 4, 128, 128, 127, 80, True, True, 2 ** 40),
]


@pytest.mark.parametrize("dtype,Hq,Hkv,d,P,n,rotary,inter,fused,pos0", CASES)
def test_append_matches_definition(dtype, Hq, Hkv, d, P, n, rotary, inter, fused, pos0):
    dt, kind = DT[dtype]
    q, k, v = _rows(n, (Hq, Hkv, Hkv), d, dt, fused, n)
    inv = _inv_freq(rotary)
    pages = -(-n // P)
    pool = B.pkv_pool_create(P, Hkv, Hq, d, kind, pages + 2)
    try:
        seq = B.pkv_seq_create(pool)
        st = torch.cuda.current_stream()
        # Old gradients in the pages: a fresh page must start at zero again.
        B.pkv_append(seq, k.contiguous(), v.contiguous(), n, st)
        ones = torch.ones(n, Hkv, d, device="cuda")
        B.pkv_grad_accumulate(seq, 0, n, ones, ones, st)
        B.pkv_seq_reset(seq)
        order = list(range(pages))[::-1]
        B.pkv_set_block_table(seq, order)
        q_out = torch.full((n, Hq, d), float("nan"), dtype=dt, device="cuda")
        B.pkv_append_rope(seq, q, q_out, k, v, n, B.rope(inv.cuda(), pos0=pos0, interleaved=inter), st)
        assert B.pkv_seq_length(seq) == n
        kg, vg = (torch.empty(n, Hkv, d, dtype=dt, device="cuda") for _ in range(2))
        dk, dv = (torch.empty(n, Hkv, d, device="cuda") for _ in range(2))
        rep = torch.empty(pages, Hkv, d, device="cuda")
        B.pkv_gather(seq, kg, vg, dk, dv, rep, st)
        B.pkv_check(pool)
        pos = np.arange(n) + pos0
        _close(q_out, *_turn(_f64(q), inv, pos, inter), dt)
        _close(kg, *_turn(_f64(k), inv, pos, inter), dt)
        assert torch.equal(vg, v)
        assert not dk.any() and not dv.any()
        # The representative averages the stored keys: at most P fp32 additions.
        stored = _f64(kg)
        err = np.abs(_f64(rep) - _reps(stored, P))
        assert (err <= (P + 2) * 2.0 ** -24 * _reps(np.abs(stored), P)).all()
    finally:
        B.pkv_pool_destroy(pool)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_appends_in_pieces_equal_one_append(dtype):
    """Partial pages completed later, positions counting from zero in each document."""
    dt, kind = DT[dtype]
    n, P, Hq, Hkv, d = 300, 128, 4, 2, 64
    q, k, v = _rows(n, (Hq, Hkv, Hkv), d, dt, True, 3)
    inv = _inv_freq(d).cuda()
    pos = torch.cat([torch.arange(70), torch.arange(230)]).cuda()
    out = []
    for cuts in ([0, 300], [0, 1, 5, 128, 129, 290, 300]):
        pool = B.pkv_pool_create(P, Hkv, Hq, d, kind, 3)
        try:
            seq = B.pkv_seq_create(pool)
            q_out = torch.empty(n, Hq, d, dtype=dt, device="cuda")
            for a, b in zip(cuts, cuts[1:]):
                B.pkv_append_rope(seq, q[a:b], q_out[a:b], k[a:b], v[a:b], b - a, B.rope(inv, positions=pos[a:b]),
                                  torch.cuda.current_stream())
            kg, vg = (torch.empty(n, Hkv, d, dtype=dt, device="cuda") for _ in range(2))
            rep = torch.empty(3, Hkv, d, device="cuda")
            B.pkv_gather(seq, kg, vg, None, None, rep, torch.cuda.current_stream())
            B.pkv_check(pool)
            out.append((q_out, kg, vg))
            stored = _f64(kg)
            assert (np.abs(_f64(rep) - _reps(stored, P)) <= (P + 2) * 2.0 ** -24 * _reps(np.abs(stored), P)).all()
        finally:
            B.pkv_pool_destroy(pool)
    for a, b in zip(*out):
        assert torch.equal(a, b)
    _close(out[0][1], *_turn(_f64(k), inv.cpu(), pos.cpu().numpy(), False), dt)


def test_no_rotation_stores_what_the_plain_append_stores():
    n, P, Hkv, d = 200, 128, 2, 128
    k, v = _rows(n, (Hkv, Hkv), d, torch.bfloat16, False, 9)
    got = []
    for rope in (None, B.rope(torch.zeros(d // 2, device="cuda"))):
        pool = B.pkv_pool_create(P, Hkv, 4, d, B.PKV_BF16, 2)
        try:
            seq = B.pkv_seq_create(pool)
            if rope is None:
                B.pkv_append(seq, k, v, n)
            else:
                B.pkv_append_rope(seq, None, None, k, v, n, rope)
            kg, vg = (torch.empty(n, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            B.pkv_gather(seq, kg, vg)
            torch.cuda.synchronize()
            got.append((kg, vg))
        finally:
            B.pkv_pool_destroy(pool)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype,Hq,Hkv,d,P,total,row0,n,rotary,inter,fused", [
    ("bf16", 28, 4, 128, 128, 300, 0, 300, 128, False, True),
    ("bf16", 6, 2, 64, 16, 100, 37, 1, 64, True, False),
    ("bf16", 14, 2, 64, 128, 260, 100, 131, 32, False, True),
    ("f32", 2, 1, 64, 16, 90, 15, 70, 64, False, True),
    ("f32", 4, 2, 128, 64, 130, 1, 129, 96, True, False),
])
def test_gradient_matches_definition(dtype, Hq, Hkv, d, P, total, row0, n, rotary, inter, fused):
    dt, kind = DT[dtype]
    pages = -(-total // P)
    pool = B.pkv_pool_create(P, Hkv, Hq, d, kind, pages + 1)
    try:
        seq = B.pkv_seq_create(pool)
        st = torch.cuda.current_stream()
        B.pkv_set_block_table(seq, list(range(pages))[::-1])
        z = torch.zeros(total, Hkv, d, dtype=dt, device="cuda")
        B.pkv_append(seq, z, z, total, st)
        dk, dv = _rows(total, (Hkv, Hkv), d, torch.float32, False, 5)
        B.pkv_grad_accumulate(seq, 0, total, dk, dv, st)
        dq, = _rows(n, (Hq,), d, dt, False, 6)
        H = Hq + 2 * Hkv
        whole = torch.full((n + 2, H + 1, d), 7.0, dtype=dt, device="cuda")     # rows and columns around the outputs
        out = whole[1:n + 1, :H].split([Hq, Hkv, Hkv], dim=1) if fused else tuple(
            torch.empty(n, h, d, dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
        inv = _inv_freq(rotary)
        B.pkv_rope_grad(seq, row0, n, B.rope(inv.cuda(), pos0=row0 + 11, interleaved=inter), dq, *out, st)
        B.pkv_check(pool)
        pos = np.arange(n) + row0 + 11
        _close(out[0], *_turn(_f64(dq), inv, pos, inter, -1), dt)
        _close(out[1], *_turn(_f64(dk[row0:row0 + n]), inv, pos, inter, -1), dt)
        assert torch.equal(out[2], dv[row0:row0 + n].to(dt))
        if fused:
            assert (whole[0] == 7).all() and (whole[-1] == 7).all() and (whole[:, H] == 7).all()
        # Parts alone: the same values; what is not asked for is not written.
        only = torch.empty(n, Hkv, d, dtype=dt, device="cuda")
        B.pkv_rope_grad(seq, row0, n, B.rope(inv.cuda(), pos0=row0 + 11, interleaved=inter), dk_out=only, stream=st)
        assert torch.equal(only, out[1])
    finally:
        B.pkv_pool_destroy(pool)


def test_gradient_is_the_adjoint_and_follows_differences():
    """<w, turn(k)> differentiated by k: the returned gradient against the inner
    products (the map is linear, so a difference quotient is exact up to
    rounding): sums of N = n Hkv d fp32-rounded terms, each within ROT."""
    n, Hkv, d, P = 40, 2, 64, 16
    pool = B.pkv_pool_create(P, Hkv, 4, d, B.PKV_F32, 3)
    try:
        seq = B.pkv_seq_create(pool)
        k, v, w = _rows(n, (Hkv, Hkv, Hkv), d, torch.float32, False, 12)
        rope = B.rope(_inv_freq(d).cuda(), pos0=1000)
        B.pkv_append_rope(seq, None, None, k, v, n, rope)
        kr = torch.empty_like(k)
        B.pkv_gather(seq, kr)
        B.pkv_grad_accumulate(seq, 0, n, w, None)
        dk = torch.empty_like(k)
        B.pkv_rope_grad(seq, 0, n, rope, dk_out=dk)
        a, b = (w.double() * kr.double()).sum().item(), (dk.double() * k.double()).sum().item()
        size = (w.abs().double() * kr.abs().double()).sum().item() * 4
        assert abs(a - b) <= 2 * ROT * size
        # One element moved by h: <w, turn(k + h e)> - <w, turn(k)> = h dk.
        for at in ((0, 0, 0), (17, 1, 40), (39, 1, 63)):
            k2, h = k.clone(), 0.5
            k2[at] += h
            B.pkv_seq_reset(seq)
            B.pkv_append_rope(seq, None, None, k2, v, n, rope)
            kr2 = torch.empty_like(k)
            B.pkv_gather(seq, kr2)
            diff = (w.double() * (kr2.double() - kr.double())).sum().item() / h
            t, hh, _ = at
            # two rounded rows of d values of size |k| + h enter the difference
            bound = 2 * ROT * (w[t, hh].abs().double() * 2 * (k[t, hh].abs().double().max() + h)).sum().item() / h
            assert abs(diff - dk[at].item()) <= bound
    finally:
        B.pkv_pool_destroy(pool)


def test_rows_in_place_and_back():
    pool = B.pkv_pool_create(16, 1, 2, 128, B.PKV_F32, 1)
    try:
        x = torch.randn(33, 12, 128, device="cuda")
        part = x[:, 3:8]                                   # 5 heads of 12, rows apart
        keep, before = x.clone(), part.clone()
        rope = B.rope(_inv_freq(96).cuda(), pos0=77)
        B.pkv_rope_rows(pool, part, part, 33, 5, rope)
        torch.cuda.synchronize()
        _close(part, *_turn(_f64(before), _inv_freq(96), np.arange(33) + 77, False), torch.float32)
        assert torch.equal(x[:, :3], keep[:, :3]) and torch.equal(x[:, 8:], keep[:, 8:])
        B.pkv_rope_rows(pool, part, part, 33, 5, rope, inverse=True)
        torch.cuda.synchronize()
        # forth and back: each turn within its bound of pairs no longer than sqrt(2) of the first
        _, mag = _turn(_f64(before), _inv_freq(96), np.arange(33) + 77, False)
        assert (np.abs(_f64(part) - _f64(before)) <= 4 * (ROT + 2.0 ** -23) * mag).all()
    finally:
        B.pkv_pool_destroy(pool)


def test_pinned_host_pool():
    """Pages in pinned host memory: keys, recorded zero gradients, added ones."""
    n, P, Hq, Hkv, d = 150, 128, 4, 2, 128
    q, k, v = _rows(n, (Hq, Hkv, Hkv), d, torch.bfloat16, True, 21)
    inv = _inv_freq(d)
    pool = B.pkv_pool_create(P, Hkv, Hq, d, B.PKV_BF16, 4, residency=B.PKV_RES_PINNED_HOST, n_device_slots=2)
    try:
        seq = B.pkv_seq_create(pool)
        q_out = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda")
        rope = B.rope(inv.cuda())
        B.pkv_append_rope(seq, q, q_out, k, v, n, rope)
        kg = torch.empty(n, Hkv, d, dtype=torch.bfloat16, device="cuda")
        dk = torch.ones_like(kg)
        B.pkv_gather(seq, kg)
        B.pkv_rope_grad(seq, 0, n, rope, dk_out=dk)
        torch.cuda.synchronize()
        _close(kg, *_turn(_f64(k), inv, np.arange(n), False), torch.bfloat16)
        assert not dk.any()
        g = torch.randn(n, Hkv, d, device="cuda")
        B.pkv_grad_accumulate(seq, 0, n, g, g)
        B.pkv_rope_grad(seq, 0, n, rope, dk_out=dk)
        B.pkv_check(pool)
        _close(dk, *_turn(_f64(g), inv, np.arange(n), False, -1), torch.bfloat16)
    finally:
        B.pkv_pool_destroy(pool)


def test_side_stream_and_captured_graph():
    """The row calls on a stream of their own and replayed from a graph with new
    inputs; an append refuses to be captured."""
    n, Hq, Hkv, d, P = 64, 4, 2, 64, 16
    pool = B.pkv_pool_create(P, Hkv, Hq, d, B.PKV_F32, 4)
    try:
        seq = B.pkv_seq_create(pool)
        x, k, v = _rows(n, (Hq, Hkv, Hkv), d, torch.float32, False, 30)
        rope = B.rope(_inv_freq(d).cuda())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out, dk = torch.empty_like(x), torch.empty_like(k)
        with torch.cuda.stream(side):
            B.pkv_append_rope(seq, None, None, k, v, n, rope, side)
            B.pkv_grad_accumulate(seq, 0, n, k, v, side)
            B.pkv_rope_rows(pool, x, out, n, Hq, rope, stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            with pytest.raises(B.PkvError) as e:
                B.pkv_append_rope(seq, None, None, k, v, n, rope, side)
            assert e.value.status == B.PKV_ERR_INVALID and "captured" in str(e.value)
            B.pkv_rope_rows(pool, x, out, n, Hq, rope, stream=side)
            B.pkv_rope_grad(seq, 0, n, rope, dk_out=dk, stream=side)
        assert B.pkv_seq_length(seq) == n
        for seed in (1, 2):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
            g.replay()
            torch.cuda.synchronize()
            _close(out, *_turn(_f64(x), _inv_freq(d), np.arange(n), False), torch.float32)
            _close(dk, *_turn(_f64(k), _inv_freq(d), np.arange(n), False, -1), torch.float32)
    finally:
        B.pkv_pool_destroy(pool)


def test_empty_calls_change_nothing():
    pool = B.pkv_pool_create(16, 1, 2, 64, B.PKV_F32, 2)
    try:
        seq = B.pkv_seq_create(pool)
        rope = B.rope(_inv_freq(64).cuda())
        e = torch.empty(0, 1, 64, device="cuda")
        B.pkv_append_rope(seq, None, None, e, e, 0, rope)
        B.pkv_rope_rows(pool, e, e, 0, 1, rope)
        B.pkv_rope_grad(seq, 0, 0, rope, dk_out=e)
        assert B.pkv_seq_length(seq) == 0 and B.pkv_pool_free_pages(pool) == 2
        x = torch.zeros(33, 1, 64, device="cuda")
        with pytest.raises(B.PkvError) as err:                 # one page too many: nothing is claimed
            B.pkv_append_rope(seq, None, None, x, x, 33, rope)
        assert err.value.status == B.PKV_ERR_OOM
        assert B.pkv_seq_length(seq) == 0 and B.pkv_pool_free_pages(pool) == 2
    finally:
        B.pkv_pool_destroy(pool)


def _turns(f, pos, bits=400):
    """pos * f / (2 pi) modulo one turn, from integers: f's own 24 bits and pi to
    `bits` bits by Machin's formula."""
    def atan_inv(x):
        one, total, term, k = 1 << bits, 0, (1 << bits) // x, 0
        while term:
            total += (term // (2 * k + 1)) * (-1) ** k
            term //= x * x
            k += 1
        return total
    two_pi = 8 * (4 * atan_inv(5) - atan_inv(239))
    num, den = float(f).as_integer_ratio()
    x = pos * num * (1 << (2 * bits)) // (den * two_pi)
    return (x % (1 << bits)) / float(1 << bits)


@pytest.mark.parametrize("pos0", [2 ** 44 + 12345, -(2 ** 47) - 1, 2 ** 50 - 3])
@pytest.mark.parametrize("theta", [1e4, 1e6])
def test_far_positions_within_half_a_unit(pos0, theta):
    """A pair's frequency is a 64-bit fraction of a turn, rounded to nearest: the
    phase is off by |p| 2^-65 turns at most, on top of the rest of ROT."""
    n, d = 9, 128
    inv = _inv_freq(d, theta)
    pool = B.pkv_pool_create(16, 1, 1, d, B.PKV_F32, 1)
    try:
        x = _rows(n, (1,), d, torch.float32, False, 55)[0]
        out = torch.empty_like(x)
        B.pkv_rope_rows(pool, x, out, n, 1, B.rope(inv.cuda(), pos0=pos0))
        torch.cuda.synchronize()
        a, b = _f64(x)[:, 0, :d // 2], _f64(x)[:, 0, d // 2:]
        ang = 2 * math.pi * np.array([[_turns(f, pos0 + t) for f in inv.tolist()] for t in range(n)])
        c, s = np.cos(ang), np.sin(ang)
        size = np.hypot(a, b)
        tol = 2 * math.pi * abs(pos0) * 2.0 ** -65 * size + (ROT + 2.0 ** -23) * (np.abs(a) + np.abs(b))
        got = _f64(out)[:, 0]
        assert (np.abs(got[:, :d // 2] - (a * c - b * s)) <= tol).all()
        assert (np.abs(got[:, d // 2:] - (b * c + a * s)) <= tol).all()
    finally:
        B.pkv_pool_destroy(pool)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_frequency_that_is_not_finite_gives_nan(dtype, bad):
    """In its own pair, whatever the position; the other pairs keep their values."""
    dt, kind = DT[dtype]
    n, Hq, Hkv, d, P = 20, 3, 1, 64, 16
    inv = _inv_freq(d)
    inv[5] = bad
    q, k, v = _rows(n, (Hq, Hkv, Hkv), d, dt, True, 60)
    pool = B.pkv_pool_create(P, Hkv, Hq, d, kind, 2)
    try:
        seq, rope = B.pkv_seq_create(pool), B.rope(inv.cuda())
        out, back = torch.empty(n, Hq, d, dtype=dt, device="cuda"), torch.empty(n, Hq, d, dtype=dt, device="cuda")
        B.pkv_append_rope(seq, q, out, k, v, n, rope)
        kg, vg, dk = (torch.empty(n, Hkv, d, dtype=dt, device="cuda") for _ in range(3))
        B.pkv_gather(seq, kg, vg)
        B.pkv_rope_rows(pool, q, back, n, Hq, rope, inverse=True)
        g = torch.randn(n, Hkv, d, device="cuda")
        B.pkv_grad_accumulate(seq, 0, n, g, g)
        B.pkv_rope_grad(seq, 0, n, rope, dk_out=dk)
        torch.cuda.synchronize()
        assert torch.equal(vg, v)
        fine = _inv_freq(d)
        fine[5] = 0.0
        pair = np.zeros(d, dtype=bool)
        pair[[5, d // 2 + 5]] = True
        for got, x, sign in ((out, q, 1), (kg, k, 1), (back, q, -1), (dk, g, -1)):
            got = _f64(got)
            assert np.isnan(got[..., pair]).all()
            want, mag = _turn(_f64(x), fine, np.arange(n), False, sign)
            tol = ROT * mag + (torch.finfo(dt).eps / 2) * (np.abs(want) + ROT * mag)
            assert (np.abs(got - want) <= tol)[..., ~pair].all()
    finally:
        B.pkv_pool_destroy(pool)
