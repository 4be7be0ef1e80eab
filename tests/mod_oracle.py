"""Attention with modified scores in float64, from the definition, with the
error bounds that rounding allows the kernels. Test infrastructure only."""
import numpy as np


def attention(q, k, v, q_start, cap=0.0, slopes=None, k_begin=None, k_end=None, listed=None, dout=None):
    """q [n, Hq, d], k, v [L, Hkv, d] float64. listed: bool [n, Hkv, L], the keys of
    the selected pages. Returns a dict of o, lse, and with dout the gradients;
    every array of weights is [Hq, n, L]."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    g = Hq // Hkv
    i = q_start + np.arange(n)
    j = np.arange(L)
    lo = np.zeros(n, dtype=np.int64) if k_begin is None else np.maximum(k_begin, 0)
    hi = i + 1 if k_end is None else np.minimum(k_end, L)
    seen = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
    out = {"o": np.zeros_like(q), "lse": np.full((Hq, n), -np.inf), "p": np.zeros((Hq, n, L)), "f": np.ones((Hq, n, L))}
    if dout is not None:
        out.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), ds=np.zeros((Hq, n, L)))
    for h in range(Hq):
        kk, vv = k[:, h // g], v[:, h // g]
        vis = seen & listed[:, h // g] if listed is not None else seen
        s = q[:, h] @ kk.T / np.sqrt(d)
        f = np.ones_like(s)
        if cap:
            t = np.tanh(s / cap)
            s, f = cap * t, 1 - t * t
        if slopes is not None:
            s = s - slopes[h] * np.abs(i[:, None] - j[None])
        s = np.where(vis, s, -np.inf)
        rows = vis.any(1)
        m = np.where(rows, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - m[:, None])
        z = e.sum(1)
        p = e / np.where(rows, z, 1.0)[:, None]
        out["lse"][h, rows] = (m + np.log(np.where(rows, z, 1.0)))[rows]
        out["o"][:, h], out["p"][h], out["f"][h] = p @ vv, p, f
        if dout is not None:
            dp = dout[:, h] @ vv.T
            ds = p * (dp - (dout[:, h] * out["o"][:, h]).sum(1, keepdims=True)) * f
            out["ds"][h] = ds
            out["dq"][:, h] = ds @ kk / np.sqrt(d)
            out["dk"][:, h // g] += ds.T @ q[:, h] / np.sqrt(d)
            out["dv"][:, h // g] += p.T @ dout[:, h]
    return out


def bounds(r, q, k, v, q_start, bf16, cap=0.0, slopes=None, dout=None, **_):
    """Largest errors that rounding explains, element by element.

    u: half an eps of the storage type (2^-8 for bf16, 2^-24 for fp32): outputs
    and, on the bf16 path, each weight P and dS before its product are rounded
    once. Logits are fp32 sums of d products, then the cap (absolute error of
    tanh below 4e-7) and the bias; sums over L keys add L 2^-24 relative to the
    sum of magnitudes."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    g, u, w = Hq // Hkv, 2.0 ** -8 if bf16 else 2.0 ** -24, 2.0 ** -8 if bf16 else 0.0
    f32, scale = 2.0 ** -24, 1 / np.sqrt(d)
    b = {"o": np.zeros_like(q), "lse": np.zeros((Hq, n))}
    if dout is not None:
        b.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    far = q_start + n + L
    for h in range(Hq):
        kk, vv = np.abs(k[:, h // g]), np.abs(v[:, h // g])
        qh = np.abs(q[:, h])
        # error of one logit, and of one weight relative to itself
        e_s = (d + 8) * f32 * (qh @ kk.T * scale).max(1, initial=0.0) + cap * 4e-7
        if slopes is not None:
            e_s = e_s + 4 * f32 * abs(slopes[h]) * far
        lse = np.where(np.isfinite(r["lse"][h]), np.abs(r["lse"][h]), 0.0)
        b["lse"][h] = e_s + (L + 8) * f32 + 8 * f32 * (lse + 1)
        e_p = (2 * e_s + (L + 16) * f32 + 2.0 ** -21)[:, None]
        A = r["p"][h] @ vv
        b["o"][:, h] = (2 * w + e_p) * A + (u + 4 * f32) * np.abs(r["o"][:, h])
        if dout is None:
            continue
        do = np.abs(dout[:, h])
        e_b = (e_s + b["lse"][h] + 16 * f32 * (lse + 1) + 2.0 ** -21)[:, None]   # P recomputed from LSE
        e_D = ((do * b["o"][:, h]).sum(1) + d * f32 * (do * A).sum(1))[:, None]
        p, f, ds = r["p"][h], np.abs(r["f"][h]), np.abs(r["ds"][h])
        e_dp = (d + 8) * f32 * (do @ vv.T)
        e_f = 1e-6 if cap else 0.0
        e_ds = (w + e_b + 8 * f32) * ds + p * f * (e_D + e_dp) + p * e_f * (do @ vv.T + (do * A).sum(1)[:, None])
        acc = (L + 16) * f32
        b["dq"][:, h] = scale * ((e_ds + acc * ds) @ kk) + (u + 4 * f32) * np.abs(r["dq"][:, h])
        acc = (n * g + 16) * f32
        b["dk"][:, h // g] += scale * ((e_ds + acc * ds).T @ qh)
        b["dv"][:, h // g] += ((w + e_b + acc) * p).T @ do
    return {name: x + 1e-30 for name, x in b.items()}
