"""The float64 oracle of linear attention and layer norm against finite
differences and against the sum over pairs of tokens. CPU only."""
import numpy as np
import pytest

import lin_oracle as O


def _inputs(n, Hq, Hkv, d, seed):
    r = np.random.default_rng(seed)
    shapes = ((n, Hq, d), (n, Hkv, d), (n, Hkv, d), (n, Hq, d), (Hkv, d, d), (Hkv, d, d))
    return [r.standard_normal(s) for s in shapes]


@pytest.mark.parametrize("n,Hq,Hkv,d", [(1, 2, 1, 3), (7, 4, 2, 4), (5, 3, 3, 2)])
def test_forward_is_the_sum_over_pairs(n, Hq, Hkv, d):
    q, k, v, _, first, _ = _inputs(n, Hq, Hkv, d, n)
    decay = np.linspace(0.5, 1.0, Hkv)
    o, last = O.lin_forward(q, k, v, decay, first)
    for h in range(Hq):
        x = h // (Hq // Hkv)
        for i in range(n):
            want = decay[x] ** (i + 1) * (q[i, h] @ first[x])
            for j in range(i + 1):
                want = want + decay[x] ** (i - j) * (q[i, h] @ k[j, x]) * v[j, x]
            np.testing.assert_allclose(o[i, h], want / np.sqrt(d), rtol=1e-12, atol=1e-12)
    want = decay[:, None, None] ** n * first + sum(decay[:, None, None] ** (n - 1 - j) * k[j][:, :, None] * v[j][:, None, :]
                                                  for j in range(n))
    np.testing.assert_allclose(last, want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("n,Hq,Hkv,d", [(1, 2, 1, 3), (6, 4, 2, 3)])
def test_backward_against_differences(n, Hq, Hkv, d):
    q, k, v, do, first, dlast = _inputs(n, Hq, Hkv, d, 5 + n)
    decay = np.linspace(0.3, 0.95, Hkv)
    grads = O.lin_backward(q, k, v, do, decay, first, dlast)

    def loss():
        o, last = O.lin_forward(q, k, v, decay, first)
        return (o * do).sum() + (last * dlast).sum()

    for x, g in zip((q, k, v, first), grads):
        for at in np.ndindex(x.shape):
            keep, h = x[at], 1e-5
            x[at] = keep + h
            up = loss()
            x[at] = keep - h
            down = loss()
            x[at] = keep
            # Central difference of a polynomial that is quadratic at most in one entry: exact but for rounding.
            assert abs((up - down) / (2 * h) - g[at]) < 1e-8 * (1 + abs(g[at]) + abs(up))


def test_norm_against_differences():
    r = np.random.default_rng(2)
    x, dy = r.standard_normal((3, 2, 5)), r.standard_normal((3, 2, 5))
    w, b = r.standard_normal((2, 5)), r.standard_normal((2, 5))
    _, mean, rstd = O.norm_forward(x, w, b, 1e-3)
    grads = O.norm_backward(dy, x, w, mean, rstd)
    for t, g in zip((x, w, b), grads):
        for at in np.ndindex(t.shape):
            keep, h = t[at], 1e-5
            t[at] = keep + h
            up = (O.norm_forward(x, w, b, 1e-3)[0] * dy).sum()
            t[at] = keep - h
            down = (O.norm_forward(x, w, b, 1e-3)[0] * dy).sum()
            t[at] = keep
            assert abs((up - down) / (2 * h) - g[at]) < 1e-7 * (1 + abs(g[at]))
