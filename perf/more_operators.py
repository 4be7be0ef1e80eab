"""Cases that measure linear attention with a decay per head, and layer norm.

The mixer and the normalisation of a recurrent block:

* linear attention, S_t = l S_{t-1} + k_t v_t^T, o_t = q_t^T S_t / sqrt(d), one
  decay l for each KV head, query heads in groups: the rows of a call are packed
  sequences, each with a state that it starts from and one that it ends with;
  forward ("prompt"), forward plus backward ("train") and one token for each of a
  batch of running sequences ("step");
* layer norm of whole rows or of each head of a row, forward ("norm") and forward
  plus backward with the weight's and bias's gradients ("norm_train").

With ``own`` false the operators are computed in plain torch operations; with
``own`` true by the library's calls.
"""
import math
import random

import torch

own = False

HEADS = {"28x4x128": (28, 4, 128), "64x8x64": (64, 8, 64), "14x2x64": (14, 2, 64), "7x1x128": (7, 1, 128),
         "2x1x64": (2, 1, 64), "4x2x128": (4, 2, 128), "8x2x64": (8, 2, 64), "16x16x128": (16, 16, 128)}
EPS = 1e-5
BLOCK = 64  # rows that the plain form takes at once


# ---------------------------------------------------------------- cases

def _lin(name, op, heads, n, seqs=1, dtype="bf16", fused=True, pad=0, decay="spread", start=True):
    c = {"op": op, "heads": heads, "dtype": dtype, "n": n, "seqs": seqs, "fused": fused, "pad": pad, "decay": decay, "start": start}
    return dict(c, name=name) if name else c


def _norm(name, op, n, width, groups=1, dtype="bf16", weights="same", bias=True, gap=0):
    c = {"op": op, "n": n, "width": width, "groups": groups, "dtype": dtype, "weights": weights, "bias": bias, "gap": gap}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One generated token of one sequence: latency alone.
        _lin("one token", "step", "28x4x128", 1),
        # A full decoding batch, some of its rows padding: every state is read and written once.
        _lin("decoding batch", "step", "28x4x128", 192, pad=5),
        # A training chunk of packed documents, the first of them carried on from the chunk before.
        _lin("chunk of documents", "prompt", "28x4x128", 4096, seqs=5),
        # Prompts of several requests, short and long, head dimension 64, the last rows padding.
        _lin("ragged prompts", "prompt", "64x8x64", 2777, seqs=9, fused=False, pad=40),
        # A long prompt with a state for every head.
        _lin("long prompt", "prompt", "16x16x128", 32768),
        # One training chunk, forward and backward.
        _lin("training chunk", "train", "28x4x128", 4096),
        # Packed documents of odd lengths, head dimension 64, forward and backward.
        _lin("training, odd documents", "train", "14x2x64", 1777, seqs=4, pad=3),
        # fp32 at the small test geometry, forward and backward.
        _lin("fp32 small, train", "train", "2x1x64", 201, seqs=2, dtype="f32", fused=False, decay="fast"),
        # The row of one generated token.
        _norm("norm of one row", "norm", 1, 3584),
        # A training chunk at the block's hidden size.
        _norm("norm of a chunk", "norm_train", 4096, 3584),
        # Each head of the mixer's output on its own, part of a wider tensor, fp32 weights.
        _norm("norm of heads, odd", "norm_train", 777, 64, groups=14, weights="f32", bias=False, gap=256),
        # fp32 rows of an odd width, forward alone.
        _norm("fp32 odd norm", "norm", 333, 1001, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prompt", "train", "train", "step", "norm", "norm_train"])
    f32 = rng.random() < 0.2
    dtype = "f32" if f32 else "bf16"
    if op in ("norm", "norm_train"):
        if rng.random() < 0.4:
            groups, width = rng.choice([(28, 128), (64, 64), (14, 64), (7, 128), (16, 128), (3, 80)])
        else:
            groups, width = 1, _log(rng, 16, 8192) if rng.random() < 0.4 else 8 * _log(rng, 2, 1024)
        n = _log(rng, 1, max(1, min(8192, 4096 * 3584 // (groups * width))))
        return _norm(None, op, n, width, groups, dtype, rng.choice(["same", "f32", "none"]), rng.random() < 0.7, rng.choice([0, 0, 64]))
    heads = rng.choice(["2x1x64", "4x2x128", "8x2x64"] if f32 else ["28x4x128", "64x8x64", "14x2x64", "7x1x128", "16x16x128"])
    decay, start, fused = rng.choice(["spread", "spread", "none", "fast"]), rng.random() < 0.6, rng.random() < 0.6
    if op == "step":
        c = _lin(None, op, heads, _log(rng, 1, 192), 1, dtype, fused, rng.choice([0, 0, 3]), decay, True)
        c["pad"] = min(c["pad"], c["n"] - 1)
    else:
        n = _log(rng, 1, 1024 if f32 else 4096 if op == "train" else 16384)
        seqs = rng.choice([1, 1, 2, 3, 7])
        c = _lin(None, op, heads, n, seqs, dtype, fused, rng.choice([0, 0, 17]) if n > 64 else 0, decay, start)
    most = {k: max(work(x)["bytes"] for x in listed() if x["op"] == k) for k in ("prompt", "train", "step")}
    while work(c)["bytes"] > most[op]:  # no drawn case is larger than the largest listed one
        c["n"] -= c["n"] // 3
    return c


# ---------------------------------------------------------------- what a case's sizes fix

def _cuts(case):
    """First row of each sequence and the end of the last: cuts at random (equal ones leave a sequence empty), padding behind."""
    n, seqs = case["n"] - case["pad"], case["seqs"]
    r = random.Random(1009 * seqs + n)
    return [0] + sorted(r.randrange(0, n + 1) for _ in range(seqs - 1)) + [n]


def _log_decay(case):
    """Natural log of each KV head's decay: from fast to slow over the heads, 1 for all, or a few tokens' memory."""
    Hkv = HEADS[case["heads"]][1]
    if case["decay"] == "none":
        return [0.0] * Hkv
    lo, hi = (3.0, 9.0) if case["decay"] == "spread" else (0.5, 2.0)
    return [math.log1p(-2.0 ** -(lo + (hi - lo) * (h + 1) / Hkv)) for h in range(Hkv)]


def _live(case):
    """Slots of a decoding batch: one for each row but the padding ones."""
    return case["n"] - case["pad"]


def work(case):
    n, e = case["n"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        cols = case["groups"] * case["width"]
        we = {"none": 0, "same": e, "f32": 4}[case["weights"]] * (1 + case["bias"]) * cols
        if case["op"] == "norm":  # rows read, rows written
            return {"bytes": 2 * n * cols * e + we, "flops": 8 * n * cols}
        # and dy in, dx, the weight's and bias's gradients out, the row's statistics
        return {"bytes": 4 * n * cols * e + we + 8 * cols + 8 * n * case["groups"], "flops": 22 * n * cols}
    Hq, Hkv, d = HEADS[case["heads"]]
    state = 4 * Hkv * d * d
    if case["op"] == "step":  # the rows, and each state in and out
        m = _live(case)
        return {"bytes": m * ((2 * Hq + 2 * Hkv) * d * e + 2 * state), "flops": m * (3 * Hkv + 2 * Hq) * d * d}
    m = n - case["pad"]
    b = m * (2 * Hq + 2 * Hkv) * d * e + case["seqs"] * state * (2 if case["start"] else 1)
    f = 2 * m * (Hq + Hkv) * d * d
    if case["op"] == "prompt":  # Q, K, V and the first states in, O and the last states out
        return {"bytes": b, "flops": f}
    # and dO and the last states' gradients in, dQ, dK, dV and the first states' gradients out
    return {"bytes": b + m * (2 * Hq + 2 * Hkv) * d * e + 2 * case["seqs"] * state, "flops": f + 2 * m * (2 * Hq + 3 * Hkv) * d * d}


# ---------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(seed, which, shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) % (1 << 31)) + which)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _lin_inputs(case, seed):
    """Q, K, V [n, heads, d] (slices of one projection's output, or tensors of their own), dO, the states and their gradients."""
    Hq, Hkv, d = HEADS[case["heads"]]
    n, dt = case["n"], _dtype(case)
    x = _normal(seed, 1, (n, Hq + 2 * Hkv, d), dt)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    m = _live(case) if case["op"] == "step" else case["seqs"]
    first = _normal(seed, 2, (m, Hkv, d, d), torch.float32, 2.0) if case["start"] else None
    t = {"q": q, "k": k, "v": v, "first": first}
    if case["op"] == "train":
        t["dout"] = _normal(seed, 3, (n, Hq, d), dt)
        t["dlast"] = _normal(seed, 4, (m, Hkv, d, d), torch.float32, 0.5)
    return t


def _slots(case, seed):
    """The slot of each row of a decoding batch: requests come and go, so in no order; padding rows have none."""
    g = torch.Generator().manual_seed(int(seed) % (1 << 31) + 7)
    live = torch.randperm(_live(case), generator=g)
    rows = torch.cat([live, torch.full((case["pad"],), -1, dtype=torch.int64)])
    return rows[torch.randperm(case["n"], generator=g)].to(torch.int32)


def _norm_inputs(case, seed):
    n, cols, dt = case["n"], case["groups"] * case["width"], _dtype(case)
    x = (_normal(seed, 1, (n, cols + case["gap"]), torch.float32, 1.5) + _normal(seed, 2, (n, 1), torch.float32, 0.5)).to(dt)[:, :cols]
    t = {"x": x, "w": None, "b": None}
    wt = torch.float32 if case["weights"] == "f32" else dt
    if case["weights"] != "none":
        t["w"] = (1.0 + _normal(seed, 3, (cols,), torch.float32, 0.2)).to(wt)
        t["b"] = _normal(seed, 4, (cols,), wt, 0.2) if case["bias"] else None
    if case["op"] == "norm_train":
        t["dy"] = _normal(seed, 5, (n, cols), dt)
    return t


class _Memory:
    """Device memory of a store of states, as torch.as_tensor takes it."""

    def __init__(self, store, address, shape):
        self.store = store
        self.__cuda_array_interface__ = {"shape": shape, "typestr": "<f4", "data": (address, False), "version": 2}


class _Store:
    """A store of states; freed with the state that holds it."""

    def __init__(self, case, n_slots, grads):
        from paged_kv_chunk_chunked_gb300 import binding
        self.B = binding
        Hq, Hkv, d = HEADS[case["heads"]]
        kind = binding.PKV_BF16 if case["dtype"] == "bf16" else binding.PKV_F32
        self.lin = binding.pkv_lin_create(Hkv, Hq, d, kind, n_slots, grads=grads)
        at = binding.pkv_lin_arrays(self.lin)
        self.state, self.dstate = (torch.as_tensor(_Memory(self, at[x], (n_slots, Hkv, d, d)), device="cuda") if at[x] else None
                                   for x in ("state", "dstate"))

    def __del__(self):
        if getattr(self, "lin", None):
            torch.cuda.synchronize()
            self.B.pkv_lin_destroy(self.lin)


def prepare(case, seed):
    n, dt = case["n"], _dtype(case)
    s = {"case": case, "dtype": dt}
    if case["op"] in ("norm", "norm_train"):
        s.update(_norm_inputs(case, seed))
        cols, groups = case["groups"] * case["width"], case["groups"]
        s["y"] = torch.empty((n, cols), dtype=dt, device="cuda")
        s["mean"], s["rstd"] = (torch.empty((n, groups), dtype=torch.float32, device="cuda") for _ in range(2))
        if case["op"] == "norm_train":
            s["dx"] = torch.empty((n, cols), dtype=dt, device="cuda")
            s["dw"], s["db"] = (None if s[x] is None else torch.empty(cols, dtype=torch.float32, device="cuda") for x in "wb")
        if own:
            from paged_kv_chunk_chunked_gb300 import binding as B
            s["B"] = B
            s["norm"] = B.norm(case["width"], groups=groups, eps=EPS, weight=s["w"], bias=s["b"],
                               dtype=B.PKV_BF16 if case["dtype"] == "bf16" else B.PKV_F32)
            if case["op"] == "norm_train":
                s["scratch"] = torch.empty(max(1, B.pkv_layer_norm_scratch(s["norm"], n)), dtype=torch.float32, device="cuda")
        return s
    s.update(_lin_inputs(case, seed))
    Hq, Hkv, d = HEADS[case["heads"]]
    s["log_decay"] = torch.tensor(_log_decay(case), dtype=torch.float32, device="cuda")
    s["o"] = torch.zeros((n, Hq, d), dtype=dt, device="cuda")
    if case["op"] == "step":
        s["slots"] = _slots(case, seed).cuda()
        if own:
            s["store"] = _Store(case, _live(case), False)
            s["store"].state.copy_(s.pop("first"))
        return s
    m = case["seqs"]
    s["cu"] = torch.tensor(_cuts(case), dtype=torch.int64, device="cuda")
    if case["op"] == "train":
        s["dq"] = torch.zeros_like(s["o"])
        s["dk"], s["dv"] = (torch.zeros((n, Hkv, d), dtype=dt, device="cuda") for _ in range(2))
    if own:  # slots 0 .. m - 1: the first states; m .. 2 m - 1: the last ones
        c = s["store"] = _Store(case, 2 * m, case["op"] == "train")
        if case["start"]:
            c.state[:m] = s.pop("first")
        if case["op"] == "train":
            c.dstate[m:] = s.pop("dlast")
        at = torch.arange(m, dtype=torch.int32, device="cuda")
        s["batch"] = c.B.lin_batch(m, cu=s["cu"], slot_in=at, slot_out=at + m)  # (a new store's states are zero)
    return s


# ---------------------------------------------------------------- the plain forms

def _blocks(s):
    """The sequences in rows of blocks: row index and validity [m, blocks, BLOCK], rows of each block, tokens before each block (and at the end)."""
    c = s["case"]
    cuts = _cuts(c)
    most = max(max(b - a for a, b in zip(cuts, cuts[1:])), 1)
    nb = -(-most // BLOCK)
    lens = s["cu"][1:] - s["cu"][:-1]
    at = torch.arange(nb * BLOCK, device="cuda").view(nb, BLOCK)
    valid = at < lens[:, None, None]
    rows = torch.where(valid, at + s["cu"][:-1, None, None], 0)
    before = torch.minimum(torch.arange(nb + 1, device="cuda") * BLOCK, lens[:, None])
    return rows, valid, before


def _power(s, m):
    """decay ** m for each KV head, heads last; 0 where m is negative."""
    m = m[..., None].float()
    return torch.exp(s["log_decay"] * m.clamp(min=0)).masked_fill_(m < 0, 0.0)


def _gather(x, rows, valid):
    """[n, h, d] -> [m, blocks, h, BLOCK, d] float32, zero where there is no row."""
    return (x[rows].float() * valid[..., None, None]).transpose(2, 3).contiguous()


def _scatter(x, rows, valid, out):
    """The blocks' valid rows [m, blocks, h, BLOCK, d] into out [n, h, d]; the others as they were."""
    out[rows[valid]] = x.transpose(2, 3)[valid].to(out.dtype)
    return out


def _plain_lin(s):
    c = s["case"]
    Hq, Hkv, d = HEADS[c["heads"]]
    g, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    rows, valid, before = _blocks(s)
    m, nb = rows.shape[:2]
    q, k, v = (_gather(s[x], rows, valid) for x in "qkv")
    q = q.view(m, nb, Hkv, g * BLOCK, d)
    i = torch.arange(BLOCK, device="cuda")
    count = before[:, 1:] - before[:, :-1]
    to_end = _power(s, count[..., None] - 1 - i).transpose(2, 3)[..., None]              # [m, nb, Hkv, BLOCK, 1]
    from_start = _power(s, i + 1).t()[:, None, :].expand(Hkv, g, BLOCK).reshape(Hkv, g * BLOCK, 1)
    inside = _power(s, i[:, None] - i).permute(2, 0, 1)[:, None].expand(Hkv, g, BLOCK, BLOCK).reshape(Hkv, g * BLOCK, BLOCK)
    # States before each block and at the end: the first state and all earlier blocks' sums, decayed to there.
    part = torch.matmul((k * to_end).transpose(-1, -2), v)                               # [m, nb, Hkv, d, d]
    carry = _power(s, before[:, :, None] - before[:, None, 1:])                           # [m, nb + 1, nb, Hkv]
    later = torch.arange(nb + 1, device="cuda")[:, None] > torch.arange(nb, device="cuda")
    carry = (carry * later[..., None]).permute(0, 3, 1, 2)
    states = torch.matmul(carry, part.transpose(1, 2).reshape(m, Hkv, nb, d * d))         # [m, Hkv, nb + 1, d * d]
    if c["start"]:
        states += _power(s, before).transpose(1, 2)[..., None] * s["first"].view(m, Hkv, 1, d * d)
    states = states.view(m, Hkv, nb + 1, d, d).transpose(1, 2)                            # [m, nb + 1, Hkv, d, d]
    score = torch.matmul(q, k.transpose(-1, -2)) * inside
    o = (torch.matmul(score, v) + from_start * torch.matmul(q, states[:, :-1])) * scale
    heads = lambda x: x.view(m, nb, Hq, BLOCK, d)  # noqa: E731
    out = {"o": _scatter(heads(o), rows, valid, s["o"]), "state": states[:, -1].contiguous()}
    if c["op"] == "prompt":
        return out
    do = _gather(s["dout"], rows, valid).view(m, nb, Hkv, g * BLOCK, d)
    # Gradients of the states before each block: the last state's and all later blocks' sums, decayed back.
    part = torch.matmul((q * from_start).transpose(-1, -2), do) * scale
    carry = _power(s, before[:, None, :-1] - before[:, :, None])                          # [m, nb + 1, nb, Hkv]
    earlier = torch.arange(nb + 1, device="cuda")[:, None] <= torch.arange(nb, device="cuda")
    carry = (carry * earlier[..., None]).permute(0, 3, 1, 2)
    grads = torch.matmul(carry, part.transpose(1, 2).reshape(m, Hkv, nb, d * d))
    grads += _power(s, before[:, -1:] - before).transpose(1, 2)[..., None] * s["dlast"].view(m, Hkv, 1, d * d)
    grads = grads.view(m, Hkv, nb + 1, d, d).transpose(1, 2)
    dscore = torch.matmul(do, v.transpose(-1, -2)) * inside
    dq = (torch.matmul(dscore, k) + from_start * torch.matmul(do, states[:, :-1].transpose(-1, -2))) * scale
    dk = torch.matmul(dscore.transpose(-1, -2), q) * scale + to_end * torch.matmul(v, grads[:, 1:].transpose(-1, -2))
    dv = torch.matmul(score.transpose(-1, -2), do) * scale + to_end * torch.matmul(k, grads[:, 1:])
    out["dq"] = _scatter(heads(dq), rows, valid, s["dq"])
    out["dk"], out["dv"] = _scatter(dk, rows, valid, s["dk"]), _scatter(dv, rows, valid, s["dv"])
    out["dstate"] = grads[:, 0].contiguous()
    return out


def _plain_step(s):
    c = s["case"]
    Hq, Hkv, d = HEADS[c["heads"]]
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    q, k, v = (s[x][live].float() for x in "qkv")
    state = s["first"][at] * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
    s["first"][at] = state
    o = torch.matmul(q.view(len(at), Hkv, Hq // Hkv, d), state).mul_(1.0 / math.sqrt(d))
    s["o"][live] = o.view(len(at), Hq, d).to(s["dtype"])
    return {"o": s["o"], "state": s["first"]}


def _plain_norm(s):
    c = s["case"]
    n, groups, width = c["n"], c["groups"], c["width"]
    x = s["x"].float().view(n, groups, width)
    mean = x.mean(-1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * rstd
    w, b = (None if s[t] is None else s[t].float().view(groups, width) for t in "wb")
    y = x if w is None else x * w
    y = y if b is None else y + b
    s["y"].copy_(y.view(n, -1))
    out = {"y": s["y"], "mean": mean.view(n, groups), "rstd": rstd.view(n, groups)}
    if c["op"] == "norm":
        return out
    dy = s["dy"].float().view(n, groups, width)
    if w is not None:
        out["dw"] = (dy * x).sum(0).view(-1)
    if b is not None:
        out["db"] = dy.sum(0).view(-1)
    dy = dy if w is None else dy * w
    dx = (dy - dy.mean(-1, keepdim=True) - x * (dy * x).mean(-1, keepdim=True)) * rstd
    s["dx"].copy_(dx.view(n, -1))
    out["dx"] = s["dx"]
    return out


# ---------------------------------------------------------------- the library's calls

def _own_lin(s):
    c, n, stream = s["store"], s["case"]["n"], torch.cuda.current_stream()
    m = s["case"]["seqs"]
    c.B.pkv_lin_attn_fwd(c.lin, s["q"], s["k"], s["v"], s["o"], n, s["log_decay"], s["batch"], stream)
    out = {"o": s["o"], "state": c.state[m:]}
    if s["case"]["op"] == "prompt":
        return out
    c.B.pkv_lin_attn_bwd(c.lin, s["q"], s["k"], s["v"], s["dout"], s["dq"], s["dk"], s["dv"], n, s["log_decay"], s["batch"], stream)
    return dict(out, dq=s["dq"], dk=s["dk"], dv=s["dv"], dstate=c.dstate[:m])


def _own_step(s):
    c = s["store"]
    c.B.pkv_lin_attn_step(c.lin, s["q"], s["k"], s["v"], s["o"], s["case"]["n"], s["log_decay"], s["slots"], torch.cuda.current_stream())
    return {"o": s["o"], "state": c.state}


def _own_norm(s):
    B, n, stream = s["B"], s["case"]["n"], torch.cuda.current_stream()
    B.pkv_layer_norm_fwd(s["x"], s["y"], s["mean"], s["rstd"], n, s["norm"], stream)
    out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if s["case"]["op"] == "norm":
        return out
    B.pkv_layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"], n, s["norm"], s["scratch"], stream=stream)
    out["dx"] = s["dx"]
    return dict(out, **{x: s[x] for x in ("dw", "db") if s[x] is not None})


def run(state):
    op = state["case"]["op"]
    if op in ("norm", "norm_train"):
        return _own_norm(state) if own else _plain_norm(state)
    if op == "step":
        return _own_step(state) if own else _plain_step(state)
    return _own_lin(state) if own else _plain_lin(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_lin(case, seed):
    """Each sequence by itself, a few hundred tokens after another, every query head with a K and V of its own; gradients by autograd."""
    Hq, Hkv, d = HEADS[case["heads"]]
    n, g = case["n"], Hq // Hkv
    train = case["op"] == "train"
    t = {x: None if y is None else y.double() for x, y in _lin_inputs(case, seed).items()}
    q, k, v = (t[x].transpose(0, 1).contiguous().requires_grad_(train) for x in "qkv")       # [h, n, d]
    gamma = torch.tensor(_log_decay(case), dtype=torch.float32, device="cuda").double().repeat_interleave(g)
    cuts = _cuts(case)
    zero = torch.zeros((Hkv, d, d), dtype=torch.float64, device="cuda")
    firsts = [(t["first"][b] if case["start"] else zero).clone().requires_grad_(train) for b in range(case["seqs"])]
    o = torch.zeros((n, Hq, d), dtype=torch.float64, device="cuda")
    last, loss = [], 0.0
    for b, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        state = firsts[b].repeat_interleave(g, 0)
        for a in range(lo, hi, 256):
            z = min(hi, a + 256)
            i = torch.arange(z - a, device="cuda", dtype=torch.float64)
            age = i[:, None] - i
            weight = torch.where(age >= 0, torch.exp(gamma[:, None, None] * age.clamp(min=0)), 0.0)
            qb = q[:, a:z] / math.sqrt(d)
            kb, vb = (x[:, a:z].repeat_interleave(g, 0) for x in (k, v))
            ob = (qb @ kb.transpose(1, 2) * weight) @ vb + torch.exp(gamma[:, None] * (i + 1))[..., None] * (qb @ state)
            state = torch.exp(gamma * (z - a))[:, None, None] * state + (kb * torch.exp(gamma[:, None] * (z - a - 1 - i))[..., None]).transpose(1, 2) @ vb
            o[a:z] = ob.detach().transpose(0, 1)
            if train:
                loss = loss + (ob * t["dout"][a:z].transpose(0, 1)).sum()
        last.append(state.view(Hkv, g, d, d)[:, 0])          # the query heads of a group hold the same state
        if train:
            loss = loss + (last[-1] * t["dlast"][b]).sum()
    out = {"o": o, "state": torch.stack(last).detach()}
    if train:
        grads = torch.autograd.grad(loss, [q, k, v] + firsts)
        out.update(zip(("dq", "dk", "dv"), (x.transpose(0, 1) for x in grads[:3])), dstate=torch.stack(grads[3:]))
    return out


def _exact_step(case, seed):
    Hq, Hkv, d = HEADS[case["heads"]]
    t = {x: None if y is None else y.double() for x, y in _lin_inputs(case, seed).items()}
    gamma = torch.tensor(_log_decay(case), dtype=torch.float32, device="cuda").double().exp()
    state = t["first"].clone()
    o = torch.zeros((case["n"], Hq, d), dtype=torch.float64, device="cuda")
    for r, slot in enumerate(_slots(case, seed).tolist()):
        if slot >= 0:
            state[slot] = gamma[:, None, None] * state[slot] + torch.einsum("hi,hj->hij", t["k"][r], t["v"][r])
            o[r] = torch.einsum("hi,hij->hj", t["q"][r], state[slot].repeat_interleave(Hq // Hkv, 0)) / math.sqrt(d)
    return {"o": o, "state": state}


def _exact_norm(case, seed):
    n, groups, width = case["n"], case["groups"], case["width"]
    t = {x: None if y is None else y.double() for x, y in _norm_inputs(case, seed).items()}
    train = case["op"] == "norm_train"
    x = t["x"].reshape(n, groups, width).requires_grad_(train)
    w, b = (None if t[z] is None else t[z].view(groups, width).requires_grad_(train) for z in "wb")
    mean = x.sum(-1, keepdim=True) / width
    var = (x * x).sum(-1, keepdim=True) / width - mean * mean
    y = (x - mean) / torch.sqrt(var + EPS)
    y = y if w is None else y * w
    y = y if b is None else y + b
    out = {"y": y.detach().view(n, -1), "mean": mean.detach().view(n, groups), "rstd": 1.0 / torch.sqrt(var + EPS).detach().view(n, groups)}
    if train:
        leaves = {name: z for name, z in (("dx", x), ("dw", w), ("db", b)) if z is not None}
        grads = torch.autograd.grad((y.reshape(n, -1) * t["dy"]).sum(), list(leaves.values()))
        out.update((name, z.reshape(n, -1) if name == "dx" else z.reshape(-1)) for name, z in zip(leaves, grads))
    return out


def exact(case, seed):
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(case, seed)
    return _exact_step(case, seed) if case["op"] == "step" else _exact_lin(case, seed)
