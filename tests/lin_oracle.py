"""Linear attention with a decay per head, and layer norm, in float64: the
recurrences and definitions themselves, token by token and row by row. Test
infrastructure only."""
import numpy as np


def lin_forward(q, k, v, decay, first, last_only=False):
    """One sequence. q [n, Hq, d], k, v [n, Hkv, d], decay [Hkv] (not its log), first
    [Hkv, d, d] -> o, last state."""
    n, Hq, d = q.shape
    g = Hq // k.shape[1]
    S, o = first.copy(), np.zeros(q.shape)
    for t in range(n):
        S = decay[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = np.einsum("hi,hij->hj", q[t], np.repeat(S, g, 0)) / np.sqrt(d)
    return o, S


def lin_backward(q, k, v, do, decay, first, dlast):
    """Gradients dq, dk, dv, dfirst: the recurrence run backwards. The gradient of S_t is
    scale q_t do_t^T (over the group's heads) plus decay times that of S_{t+1}."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    g, scale = Hq // Hkv, 1 / np.sqrt(d)
    S, states = first.copy(), []
    for t in range(n):
        S = decay[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        states.append(S)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    G = dlast.copy()
    for t in reversed(range(n)):
        G = G + scale * np.einsum("hei,hej->hij", q[t].reshape(Hkv, g, d), do[t].reshape(Hkv, g, d))
        dq[t] = scale * np.einsum("hij,hj->hi", np.repeat(states[t], g, 0), do[t])
        dk[t] = np.einsum("hij,hj->hi", G, v[t])
        dv[t] = np.einsum("hij,hi->hj", G, k[t])
        G = decay[:, None, None] * G
    return dq, dk, dv, G


def norm_forward(x, w, b, eps):
    """x [n, groups, width], w, b [groups, width] -> y, mean, rstd [n, groups]."""
    mean = x.mean(-1)
    rstd = 1 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    return (x - mean[..., None]) * rstd[..., None] * w + b, mean, rstd


def norm_backward(dy, x, w, mean, rstd):
    """dx, dw, db by the formula, from the statistics given."""
    xhat = (x - mean[..., None]) * rstd[..., None]
    u = dy * w
    dx = rstd[..., None] * (u - u.mean(-1, keepdims=True) - xhat * (u * xhat).mean(-1, keepdims=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)
