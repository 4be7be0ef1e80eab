"""The float64 oracle of modified scores against brute force, differences and
closed forms, on the CPU."""
import numpy as np
import pytest

import mod_oracle


def _inputs(n, L, Hq, Hkv, d, seed):
    r = np.random.default_rng(seed)
    return r.normal(size=(n, Hq, d)), r.normal(size=(L, Hkv, d)), r.normal(size=(L, Hkv, d)), r.normal(size=(n, Hq, d))


CASES = [
    dict(),
    dict(cap=1.5),
    dict(slopes=np.array([0.5, 0.01])),
    dict(cap=0.7, slopes=np.array([0.3, -0.1]), k_begin=np.array([0, 2, 9, 5, 5]), k_end=np.array([4, 9, 9, 99, 6])),
]


@pytest.mark.parametrize("kw", CASES)
def test_each_weight_by_itself(kw):
    n, L, q_start, d = 5, 11, 4, 8
    q, k, v, _ = _inputs(n, L, 2, 1, d, 0)
    r = mod_oracle.attention(q, k, v, q_start, **kw)
    for h in range(2):
        for a in range(n):
            i = q_start + a
            lo = max(0, kw["k_begin"][a]) if "k_begin" in kw else 0
            hi = min(L, kw["k_end"][a]) if "k_end" in kw else i + 1
            num, den = np.zeros(d), 0.0
            for j in range(lo, hi):
                s = float(q[a, h] @ k[j, 0]) / d ** 0.5
                if kw.get("cap"):
                    s = kw["cap"] * np.tanh(s / kw["cap"])
                if "slopes" in kw:
                    s -= kw["slopes"][h] * abs(i - j)
                num, den = num + np.exp(s) * v[j, 0], den + np.exp(s)
            if hi <= lo:
                assert not r["o"][a, h].any() and r["lse"][h, a] == -np.inf
            else:
                assert np.allclose(r["o"][a, h], num / den, rtol=1e-12) and abs(r["lse"][h, a] - np.log(den)) < 1e-12


@pytest.mark.parametrize("kw", CASES)
def test_gradients_follow_differences(kw):
    n, L, q_start = 5, 11, 4
    q, k, v, w = _inputs(n, L, 2, 1, 8, 1)
    r = mod_oracle.attention(q, k, v, q_start, dout=w, **kw)
    x = {"dq": q, "dk": k, "dv": v}
    rng = np.random.default_rng(2)
    for name, a in x.items():
        step = rng.normal(size=a.shape)
        def loss(t):
            y = dict(x, **{name: a + t * step})
            return (w * mod_oracle.attention(y["dq"], y["dk"], y["dv"], q_start, **kw)["o"]).sum()
        h = 1e-4
        diff = (loss(h) - loss(-h)) / (2 * h)
        assert abs(diff - (r[name] * step).sum()) < 1e-6 * (1 + abs(diff))


def test_limits():
    q, k, v, w = _inputs(4, 9, 2, 2, 8, 3)
    plain = mod_oracle.attention(q, k, v, 5, dout=w)
    wide = mod_oracle.attention(q, k, v, 5, cap=1e6, slopes=np.zeros(2), k_begin=np.full(4, -3), k_end=np.arange(6, 10), dout=w)
    for name in ("o", "lse", "dq", "dk", "dv"):
        assert np.allclose(plain[name], wide[name], atol=1e-9)
    one = mod_oracle.attention(q, k, v, 5, k_begin=np.arange(5, 9))       # every query sees its own key alone
    assert np.allclose(one["o"], v[5:9]) 
