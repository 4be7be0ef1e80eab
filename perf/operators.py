"""Cases that measure the rotated append and the masked, capped or biased chunk attention.

Two families, each in both directions, on the paged KV cache:

* rotation: the append of a chunk's K/V to its pages with the position
  rotation applied to Q and K on the way ("append"), and the way back: dQ and
  the paged fp32 dK rotated by the opposite angle and laid out, with dV, as the
  gradient of the projections' outputs ("rope_grad");
* attention of one query chunk over the paged cache with scores capped by a
  tanh, lowered in proportion to the distance, and restricted to a range of
  keys for each query (documents, a prefix, a window), forward ("attn") and
  forward plus backward with dK/dV added into the gradient pages ("train").

With ``own`` false the operators are computed in plain torch operations; with
``own`` true by the library's calls.
"""
import math
import random

import torch

own = False

HEADS = {"28x4x128": (28, 4, 128), "64x8x64": (64, 8, 64), "14x2x64": (14, 2, 64), "7x1x128": (7, 1, 128),
         "2x1x64": (2, 1, 64), "4x2x128": (4, 2, 128), "8x2x64": (8, 2, 64)}
THETA = 1.0e6


# ---------------------------------------------------------------- cases

def _rope_case(name, op, heads, n, start=0, dtype="bf16", page=128, fused=True, rotary=None, interleaved=False, docs=0):
    c = {"op": op, "heads": heads, "dtype": dtype, "page": page, "n": n, "start": start, "fused": fused,
         "rotary": rotary or HEADS[heads][2], "interleaved": interleaved, "docs": docs}
    return dict(c, name=name) if name else c


def _attn_case(name, op, heads, n, ctx, dtype="bf16", page=128, cap=0.0, bias=False, mask="causal", docs=0):
    c = {"op": op, "heads": heads, "dtype": dtype, "page": page, "n": n, "ctx": ctx, "cap": cap, "bias": bias, "mask": mask,
         "docs": docs}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One generated token joins a cache: latency alone.
        _rope_case("append one token", "append", "28x4x128", 1, start=20011),
        # A short fp32 sequence of the small test geometry: part of the head is rotated, pairs are neighbours.
        _rope_case("append fp32 odd", "append", "2x1x64", 201, dtype="f32", page=16, fused=False, rotary=32, interleaved=True),
        # A training chunk of packed documents, Q/K/V side by side as one projection gives them.
        _rope_case("append chunk", "append", "28x4x128", 4096, docs=5),
        # The gradient rows of a ragged last chunk, head dimension 64.
        _rope_case("rotation gradient odd", "rope_grad", "14x2x64", 777, start=500, fused=False),
        # The gradient of a whole training chunk.
        _rope_case("rotation gradient chunk", "rope_grad", "28x4x128", 4096, docs=5),
        # One token against a long cache, capped scores: serving.
        _attn_case("one token, 128K cache", "attn", "28x4x128", 1, 131071, cap=50.0),
        # A few tokens at once against a cache of medium length, every key lowered by its distance, in a window.
        _attn_case("five tokens, biased window", "attn", "64x8x64", 5, 20011, bias=True, mask="window"),
        # A ragged chunk with a prefix that is seen as a whole.
        _attn_case("prefix chunk, odd", "attn", "28x4x128", 1001, 2500, mask="prefix"),
        # A training chunk of packed documents with capped scores, the last rows padding: forward alone.
        _attn_case("documents, capped", "attn", "28x4x128", 4096, 12288, cap=50.0, mask="docs", docs=3),
        # The same forward and backward.
        _attn_case("documents, capped, train", "train", "28x4x128", 4096, 12288, cap=50.0, mask="docs", docs=3),
        # Head dimension 64 with the distance bias, forward and backward.
        _attn_case("distance bias, train", "train", "64x8x64", 1024, 4096, bias=True),
        # fp32 at the small test geometry, everything at once.
        _attn_case("fp32 small, train", "train", "2x1x64", 64, 192, dtype="f32", page=16, cap=15.0, bias=True, mask="prefix"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "rope_grad", "attn", "attn", "train"])
    f32 = rng.random() < 0.2
    dtype = "f32" if f32 else "bf16"
    if op in ("append", "rope_grad"):
        heads = rng.choice(["2x1x64", "4x2x128", "8x2x64"] if f32 else ["28x4x128", "64x8x64", "14x2x64", "7x1x128"])
        d = HEADS[heads][2]
        return _rope_case(None, op, heads, _log(rng, 1, 1024 if f32 else 4096), start=_log(rng, 1, 100000) if op == "append" else _log(rng, 1, 4000),
                          dtype=dtype, page=rng.choice([16, 64, 128]), fused=rng.random() < 0.7,
                          rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3, docs=rng.choice([0, 0, 3]))
    heads = rng.choice(["2x1x64", "4x2x128", "8x2x64"] if f32 else ["28x4x128", "64x8x64", "14x2x64", "7x1x128"])
    if f32:
        n, ctx = _log(rng, 1 if op == "attn" else 16, 256), _log(rng, 16, 1024)
    elif op == "attn" and rng.random() < 0.5:
        n, ctx = _log(rng, 1, 16), _log(rng, 100, 100000)
    elif heads in ("28x4x128", "7x1x128"):
        n, ctx = _log(rng, 17 if op == "attn" else 128, 4096), _log(rng, 100, 12000)
    else:
        n, ctx = _log(rng, 17 if op == "attn" else 128, 2048), _log(rng, 100, 6000)
    mask = rng.choice(["causal", "docs", "prefix", "window"])
    c = _attn_case(None, op, heads, n, ctx, dtype=dtype, page=rng.choice([16, 64, 128]) if f32 else 128,
                   cap=rng.choice([0.0, 15.0, 30.0, 50.0]), bias=rng.random() < 0.4, mask=mask, docs=rng.choice([2, 4, 9]) if mask == "docs" else 0)
    most = max(work(x)["flops"] for x in listed())
    while work(c)["flops"] > most:  # no drawn case is larger than the largest listed one
        c["n"] -= c["n"] // 3
    return c


# ---------------------------------------------------------------- what a case's sizes fix

def _cuts(case, total):
    """First tokens of the packed documents of `total` tokens: 0 and docs - 1 cuts."""
    r = random.Random(1009 * case["docs"] + total)
    return [0] + sorted(r.sample(range(1, total), min(case["docs"] - 1, max(0, total - 1))))


def _positions(case):
    """Position of each appended token: counted on from `start`, or from the first token of its document."""
    n = case["n"]
    pos = torch.arange(n, dtype=torch.int64)
    if not case["docs"] or n < 2:
        return pos + case["start"]
    first = torch.zeros(n, dtype=torch.int64)
    for c in _cuts(case, n):
        first[c:] = c
    return pos - first


def _ranges(case):
    """[first visible key, one past the last) for each query of the chunk; None where the operator's own defaults hold."""
    n, ctx = case["n"], case["ctx"]
    total = ctx + n
    i = torch.arange(ctx, total, dtype=torch.int64)
    lo, hi = torch.zeros_like(i), i + 1
    if case["mask"] == "causal":
        return None, None
    if case["mask"] == "window":
        return torch.clamp(i + 1 - max(1, (total + 1) // 3), min=0), None
    if case["mask"] == "prefix":  # the first part of the sequence, into the chunk, is seen by all its queries
        return None, torch.maximum(hi, torch.full_like(hi, ctx + n // 3))
    first = torch.zeros(total, dtype=torch.int64)
    for c in _cuts(case, total):
        first[c:] = c
    lo = first[ctx:].clone()
    pad = min(64, n // 16)  # the chunk's last rows are padding: they see nothing
    if pad:
        lo[n - pad:], hi[n - pad:] = 0, 0
    return lo, hi


def work(case):
    Hq, Hkv, d = HEADS[case["heads"]]
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["n"]
    if case["op"] == "append":  # Q, K, V read; Q and the rows' pages written, fresh gradient pages zeroed, representatives
        pages = -(-n // case["page"])
        return {"bytes": 2 * n * (Hq + 2 * Hkv) * d * e + 8 * pages * Hkv * case["page"] * d + 4 * pages * Hkv * d,
                "flops": 3 * n * (Hq + Hkv) * case["rotary"]}
    if case["op"] == "rope_grad":  # dQ and the fp32 gradient rows read; the three gradients written
        return {"bytes": n * (2 * Hq * e + 2 * Hkv * (4 + e)) * d, "flops": 3 * n * (Hq + Hkv) * case["rotary"]}
    lo, hi = _ranges(case)
    i = torch.arange(case["ctx"], case["ctx"] + n, dtype=torch.int64)
    lo = torch.zeros_like(i) if lo is None else lo
    hi = i + 1 if hi is None else hi
    live = hi > lo
    pairs = int((hi - lo)[live].sum())
    keys = int(hi[live].max() - lo[live].min())
    b = 2 * n * Hq * d * e + 4 * n * Hq + 2 * keys * Hkv * d * e
    if case["op"] == "train":  # and dO in, dQ, dK, dV out
        return {"bytes": b + 2 * n * Hq * d * e + 2 * keys * Hkv * d * e, "flops": 14 * pairs * Hq * d}
    return {"bytes": b, "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(seed, which, shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) % (1 << 31)) + which)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _inv_freq(case):
    r = case["rotary"]
    return torch.tensor([THETA ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float32, device="cuda")


def _heads_inputs(case, seed):
    """Q, K, V [n, heads, d]: slices of one projection's output, or tensors of their own."""
    Hq, Hkv, d = HEADS[case["heads"]]
    n = case["n"]
    x = _normal(seed, 1, (n, Hq + 2 * Hkv, d), _dtype(case))
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    return (q, k, v) if case["fused"] else (q.contiguous(), k.contiguous(), v.contiguous())


def _table(n_pages, seed):
    g = torch.Generator().manual_seed(int(seed) % (1 << 31) + 7)
    return torch.randperm(n_pages, generator=g)


def _attn_inputs(case, seed):
    Hq, Hkv, d = HEADS[case["heads"]]
    n, total, dt = case["n"], case["ctx"] + case["n"], _dtype(case)
    return {"q": _normal(seed, 1, (n, Hq, d), dt, 2.0), "k": _normal(seed, 2, (total, Hkv, d), dt),
            "v": _normal(seed, 3, (total, Hkv, d), dt), "dout": _normal(seed, 4, (n, Hq, d), dt)}


def _slopes(case):
    Hq = HEADS[case["heads"]][0]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], dtype=torch.float32, device="cuda")


class _Cache:
    """A pool with one sequence; freed with the state that holds it."""

    def __init__(self, case, n_pages):
        from paged_kv_chunk_chunked_gb300 import binding
        self.B = binding
        self.Hq, self.Hkv, self.d = HEADS[case["heads"]]
        self.P, self.n_pages, self.dtype = case["page"], n_pages, _dtype(case)
        kind = binding.PKV_BF16 if case["dtype"] == "bf16" else binding.PKV_F32
        self.pool = binding.pkv_pool_create(self.P, self.Hkv, self.Hq, self.d, kind, n_pages)
        self.seq = binding.pkv_seq_create(self.pool)

    def arrays(self):
        """The pool's pages and representatives as tensors (no copies)."""
        shape = (self.n_pages, self.Hkv, self.P, self.d)
        at = self.B.pkv_pool_arrays(self.pool)
        kv = "<i2" if self.dtype == torch.bfloat16 else "<f4"
        return {n: torch.as_tensor(_Memory(self, at[n], s, kind), device="cuda").view(t) for n, s, kind, t in (
            ("k", shape, kv, self.dtype), ("v", shape, kv, self.dtype), ("dk", shape, "<f4", torch.float32),
            ("dv", shape, "<f4", torch.float32), ("rep", (self.n_pages, self.Hkv, self.d), "<f4", torch.float32))}

    def __del__(self):
        if getattr(self, "pool", None):
            torch.cuda.synchronize()
            self.B.pkv_pool_destroy(self.pool)


class _Memory:
    """Device memory of a cache, as torch.as_tensor takes it."""

    def __init__(self, cache, address, shape, kind):
        self.cache = cache
        self.__cuda_array_interface__ = {"shape": shape, "typestr": kind, "data": (address, False), "version": 2}


def prepare(case, seed):
    Hq, Hkv, d = HEADS[case["heads"]]
    n, P, dt = case["n"], case["page"], _dtype(case)
    s = {"case": case, "dtype": dt}
    if case["op"] in ("append", "rope_grad"):
        s["inv_freq"] = _inv_freq(case)
        s["positions"] = _positions(case).cuda() if case["docs"] else None
        s["start"] = case["start"]
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = _heads_inputs(case, seed)
        s["q_out"] = torch.empty((n, Hq, d), dtype=dt, device="cuda")
        if own:
            s["cache"] = _Cache(case, -(-n // P))
            s["pages"] = s["cache"].arrays()
            s["rope"] = s["cache"].B.rope(s["inv_freq"], pos0=s["start"], positions=s["positions"], interleaved=case["interleaved"])
        return s
    if case["op"] == "rope_grad":
        total = case["start"] + n  # gradients of rows start .. start + n - 1 of the sequence
        s["dq"] = _normal(seed, 1, (n, Hq, d), dt)
        dk, dv = (_normal(seed, w, (total, Hkv, d), torch.float32) for w in (2, 3))
        n_pages = -(-total // P)
        s["table"] = _table(n_pages, seed)
        if case["fused"]:
            s["out"] = torch.empty((n, Hq + 2 * Hkv, d), dtype=dt, device="cuda").split([Hq, Hkv, Hkv], dim=1)
        else:
            s["out"] = tuple(torch.empty((n, h, d), dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
        if own:
            c = s["cache"] = _Cache(case, n_pages)
            kv = torch.zeros((total, Hkv, d), dtype=dt, device="cuda")
            c.B.pkv_set_block_table(c.seq, s["table"].tolist())
            c.B.pkv_append(c.seq, kv, kv, total, torch.cuda.current_stream())
            c.B.pkv_grad_accumulate(c.seq, 0, total, dk, dv, torch.cuda.current_stream())
            s["rope"] = c.B.rope(s["inv_freq"], pos0=s["start"], positions=s["positions"], interleaved=case["interleaved"])
        else:
            s["dk_pages"], s["dv_pages"] = (_to_pages(x, s["table"], P) for x in (dk, dv))
        s["table"] = s["table"].cuda()
        return s
    x = _attn_inputs(case, seed)
    total = case["ctx"] + n
    n_pages = -(-total // P)
    s["table"] = _table(n_pages, seed)
    s["q"], s["dout"] = x["q"], x["dout"]
    lo, hi = _ranges(case)
    s["k_begin"], s["k_end"] = (None if t is None else t.cuda() for t in (lo, hi))
    s["slopes"] = _slopes(case) if case["bias"] else None
    if own:
        c = s["cache"] = _Cache(case, n_pages)
        c.B.pkv_set_block_table(c.seq, s["table"].tolist())
        c.B.pkv_append(c.seq, x["k"], x["v"], total, torch.cuda.current_stream())
        s["mod"] = c.B.score_mod(softcap=case["cap"], slopes=s["slopes"], k_begin=s["k_begin"], k_end=s["k_end"])
        s["o"] = torch.empty((n, Hq, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((Hq, n), dtype=torch.float32, device="cuda")
        if case["op"] == "train":
            s["dq"] = torch.empty_like(s["o"])
            s["dk"], s["dv"] = (torch.empty((total, Hkv, d), dtype=torch.float32, device="cuda") for _ in range(2))
    else:
        s["k_pages"], s["v_pages"] = (_to_pages(t, s["table"], P) for t in (x["k"], x["v"]))
    s["table"] = s["table"].cuda()
    return s


# ---------------------------------------------------------------- the plain forms

def _to_pages(rows, table, P):
    """[total, H, d] rows -> physical pages [pages, H, P, d] (in logical order without a table), zero behind the last row."""
    total, H, d = rows.shape
    n_pages = -(-total // P)
    full = torch.zeros((n_pages * P, H, d), dtype=rows.dtype, device=rows.device)
    full[:total] = rows
    in_order = full.view(n_pages, P, H, d).permute(0, 2, 1, 3).contiguous()
    if table is None:
        return in_order
    pages = torch.empty_like(in_order)
    pages[table.to(rows.device)] = in_order
    return pages


def _from_pages(pages, table, total):
    """The logical rows of the pages, heads first: [H, total, d]."""
    n_pages, H, P, d = pages.shape
    return pages[table].permute(1, 0, 2, 3).reshape(H, n_pages * P, d)[:, :total]


def _cos_sin(s, n):
    """[n, 1, rotary / 2] each; the angles in 64 bits, since far positions lose them in 32."""
    pos = s["positions"] if s["positions"] is not None else torch.arange(n, device="cuda") + s["start"]
    angle = pos.double()[:, None, None] * s["inv_freq"].double()
    return angle.cos().float(), angle.sin().float()


def _rotate(x, cos, sin, interleaved):
    """x [n, H, d] float32 with its first 2 * cos.shape[-1] dims rotated."""
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, dim=-1).flatten(-2) if interleaved else torch.cat(y, dim=-1)
    return torch.cat([y, rest], dim=-1)


def _plain_append(s):
    c, dt = s["case"], s["dtype"]
    n, P = c["n"], c["page"]
    Hkv, d = HEADS[c["heads"]][1:]
    cos, sin = _cos_sin(s, n)
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(dt)
    k = _rotate(s["k"].float(), cos, sin, c["interleaved"]).to(dt)
    k_pages, v_pages = _to_pages(k, None, P), _to_pages(s["v"], None, P)
    count = torch.clamp(n - P * torch.arange(-(-n // P), device="cuda"), max=P)
    rep = k_pages.float().sum(2) / count[:, None, None]
    zero = torch.zeros(k_pages.shape, dtype=torch.float32, device="cuda")
    return {"q": q, "k": k_pages, "v": v_pages, "dk": zero, "dv": zero.clone(), "rep": _rep_out(rep, dt)}


def _rep_out(rep, dt):
    """The page means in the pages' own precision: the leading half of each word for bf16 pages, whose keys were rounded to it."""
    return rep.view(torch.bfloat16)[..., 1::2] if dt == torch.bfloat16 else rep


def _plain_rope_grad(s):
    c, dt = s["case"], s["dtype"]
    n, total = c["n"], c["start"] + c["n"]
    cos, sin = _cos_sin(s, n)
    dk, dv = (_from_pages(s[p], s["table"], total)[:, c["start"]:].transpose(0, 1) for p in ("dk_pages", "dv_pages"))
    dq_out, dk_out, dv_out = s["out"]
    dq_out.copy_(_rotate(s["dq"].float(), cos, -sin, c["interleaved"]))
    dk_out.copy_(_rotate(dk, cos, -sin, c["interleaved"]))
    dv_out.copy_(dv)
    return {"dq": dq_out, "dk": dk_out, "dv": dv_out}


def _plain_attn(s):
    c, dt = s["case"], s["dtype"]
    Hq, Hkv, d = HEADS[c["heads"]]
    n, ctx, g = c["n"], c["ctx"], Hq // Hkv
    total = ctx + n
    by_group = lambda x: x.float().view(n, Hkv, g, d).permute(1, 2, 0, 3).reshape(Hkv, g * n, d)  # noqa: E731
    back = lambda x: x.view(Hkv, g, n, d).permute(2, 0, 1, 3).reshape(n, Hq, d).to(dt)  # noqa: E731
    k, v = (_from_pages(s[p], s["table"], total).float() for p in ("k_pages", "v_pages"))
    q, scale = by_group(s["q"]), 1.0 / math.sqrt(d)
    x = torch.bmm(q, k.transpose(1, 2)).mul_(scale)
    t = None
    if c["cap"]:
        t = x.div_(c["cap"]).tanh_()
        x = t * c["cap"]
    x = x.view(Hkv, g, n, total)
    i, j = torch.arange(ctx, total, device="cuda")[:, None], torch.arange(total, device="cuda")
    if c["bias"]:
        x = x - s["slopes"].view(Hkv, g, 1, 1) * (i - j).abs().float()
    lo = 0 if s["k_begin"] is None else s["k_begin"][:, None]
    hi = i + 1 if s["k_end"] is None else s["k_end"][:, None]
    x = x.masked_fill_(~((j >= lo) & (j < hi)), -math.inf)
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill_(top == -math.inf, 0.0)
    p = x.sub_(top).exp_()
    norm = p.sum(-1, keepdim=True)
    lse = (top + norm.log()).view(Hq, n)
    p = p.div_(norm.masked_fill(norm == 0, 1.0)).view(Hkv, g * n, total)
    o = torch.bmm(p, v)
    out = {"o": back(o), "lse": lse}
    if c["op"] == "attn":
        return out
    do = by_group(s["dout"])
    ds = torch.bmm(do, v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if c["cap"]:
        ds = ds.mul_(t.square_().neg_().add_(1.0))
    out["dq"] = back(torch.bmm(ds, k).mul_(scale))
    out["dk"] = torch.bmm(ds.transpose(1, 2), q).mul_(scale).transpose(0, 1).to(dt)
    out["dv"] = torch.bmm(p.transpose(1, 2), do).transpose(0, 1).to(dt)
    return out


# ---------------------------------------------------------------- the library's calls

def _own_append(s):
    c, B, n = s["cache"], s["cache"].B, s["case"]["n"]
    B.pkv_seq_reset(c.seq)
    B.pkv_append_rope(c.seq, s["q"], s["q_out"], s["k"], s["v"], n, s["rope"], torch.cuda.current_stream())
    p = s["pages"]
    return {"q": s["q_out"], "k": p["k"], "v": p["v"], "dk": p["dk"], "dv": p["dv"], "rep": _rep_out(p["rep"], s["dtype"])}


def _own_rope_grad(s):
    c, B, case = s["cache"], s["cache"].B, s["case"]
    dq_out, dk_out, dv_out = s["out"]
    B.pkv_rope_grad(c.seq, case["start"], case["n"], s["rope"], s["dq"], dq_out, dk_out, dv_out, torch.cuda.current_stream())
    return {"dq": dq_out, "dk": dk_out, "dv": dv_out}


def _own_attn(s):
    c, B, case = s["cache"], s["cache"].B, s["case"]
    n, ctx, stream = case["n"], case["ctx"], torch.cuda.current_stream()
    B.pkv_chunk_attn_mod_fwd(c.seq, s["q"], ctx, n, s["o"], s["lse"], s["mod"], None, stream)
    out = {"o": s["o"], "lse": s["lse"]}
    if case["op"] == "attn":
        return out
    B.pkv_grad_zero(c.seq, stream)
    B.pkv_chunk_attn_mod_bwd(c.seq, s["q"], s["o"], s["dout"], s["lse"], ctx, n, s["dq"], s["mod"], None, stream)
    B.pkv_gather(c.seq, dk=s["dk"], dv=s["dv"], stream=stream)
    # The K/V projections take the gradients in the pages' type.
    return dict(out, dq=s["dq"], dk=s["dk"].to(s["dtype"]), dv=s["dv"].to(s["dtype"]))


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_append(state) if op == "append" else _own_rope_grad(state) if op == "rope_grad" else _own_attn(state)
    return _plain_append(state) if op == "append" else _plain_rope_grad(state) if op == "rope_grad" else _plain_attn(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _turn(x, case, sign):
    """Each pair (a, b) of x [n, H, d] as the complex number a + ib, times e^(sign * i * position * frequency)."""
    half = case["rotary"] // 2
    freq = _inv_freq(case).double()
    angle = sign * _positions(case).cuda().double()[:, None, None] * freq
    one = torch.arange(half, device="cuda") * (2 if case["interleaved"] else 1)
    two = one + (1 if case["interleaved"] else half)
    z = torch.complex(x[..., one], x[..., two]) * torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_append(case, seed):
    n, P = case["n"], case["page"]
    Hkv, d = HEADS[case["heads"]][1:]
    q, k, v = (t.double() for t in _heads_inputs(case, seed))
    q, k = _turn(q, case, 1.0), _turn(k, case, 1.0)
    pages = -(-n // P)
    kp, vp = (torch.zeros((pages, Hkv, P, d), dtype=torch.float64, device="cuda") for _ in range(2))
    rep = torch.zeros((pages, Hkv, d), dtype=torch.float64, device="cuda")
    for p in range(pages):
        rows = slice(p * P, min(n, p * P + P))
        m = rows.stop - rows.start
        kp[p, :, :m], vp[p, :, :m] = k[rows].transpose(0, 1), v[rows].transpose(0, 1)
        rep[p] = k[rows].to(_dtype(case)).double().mean(0)
    zero = torch.zeros_like(kp)
    return {"q": q, "k": kp, "v": vp, "dk": zero, "dv": zero, "rep": rep}


def _exact_rope_grad(case, seed):
    Hq, Hkv, d = HEADS[case["heads"]]
    n, total = case["n"], case["start"] + case["n"]
    dq = _normal(seed, 1, (n, Hq, d), _dtype(case)).double()
    dk, dv = (_normal(seed, w, (total, Hkv, d), torch.float32)[case["start"]:].double() for w in (2, 3))
    return {"dq": _turn(dq, case, -1.0), "dk": _turn(dk, case, -1.0), "dv": dv}


def _exact_attn(case, seed):
    Hq, Hkv, d = HEADS[case["heads"]]
    n, ctx = case["n"], case["ctx"]
    total, g = ctx + n, Hq // Hkv
    x = {name: t.double() for name, t in _attn_inputs(case, seed).items()}
    i = torch.arange(ctx, total, device="cuda")
    lo, hi = _ranges(case)
    lo = torch.zeros_like(i) if lo is None else lo.cuda()
    hi = i + 1 if hi is None else hi.cuda()
    j = torch.arange(total, device="cuda")
    hidden = (j[None] < lo[:, None]) | (j[None] >= hi[:, None])
    slopes = _slopes(case).double()
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"o": new(n, Hq, d), "lse": new(Hq, n)}
    if case["op"] == "train":
        out.update(dq=new(n, Hq, d), dk=new(total, Hkv, d), dv=new(total, Hkv, d))
    for h in range(Hq):
        k, v, q = x["k"][:, h // g], x["v"][:, h // g], x["q"][:, h] / math.sqrt(d)
        s = q @ k.T
        slope = 1.0
        if case["cap"]:
            u = torch.tanh(s / case["cap"])
            s, slope = case["cap"] * u, 1.0 - u * u
        if case["bias"]:
            s = s - slopes[h] * (i[:, None] - j[None]).abs()
        s[hidden] = -math.inf
        lse = torch.logsumexp(s, dim=1)
        p = torch.exp(s - lse[:, None])
        p[hidden] = 0.0
        out["o"][:, h], out["lse"][h] = p @ v, lse
        if case["op"] == "train":
            do = x["dout"][:, h]
            dp = do @ v.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * slope
            out["dq"][:, h] = ds @ k / math.sqrt(d)
            out["dk"][:, h // g] += ds.T @ q
            out["dv"][:, h // g] += p.T @ do
    return out


def exact(case, seed):
    op = case["op"]
    return _exact_append(case, seed) if op == "append" else _exact_rope_grad(case, seed) if op == "rope_grad" else _exact_attn(case, seed)
