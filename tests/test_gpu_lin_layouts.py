"""Linear attention into slices of wider tensors, and in calls of exactly the sequences' rows:
outputs are the dense call's bits, and nothing beside them is written."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from test_gpu_lin import DT, Store, _decays, _lib, _rows  # noqa: F401

pytestmark = pytest.mark.gpu


def _both(c, x, outs, n, g2, batch):
    st = torch.cuda.current_stream()
    B.pkv_lin_attn_fwd(c.lin, *x[:3], outs[0], n, g2, batch, st)
    B.pkv_lin_attn_bwd(c.lin, *x, *outs[1:], n, g2, batch, st)
    B.pkv_lin_check(c.lin)


@pytest.mark.parametrize("flags", [0, B.PKV_FLAG_LIN_ONE_TERM])
@pytest.mark.parametrize("dtype,Hq,Hkv,d,n,cuts", [
    ("bf16", 4, 2, 128, 300, [0, 300]), ("bf16", 6, 2, 64, 385, [5, 133, 140, 380]), ("bf16", 1, 1, 64, 1, [0, 1]),
    ("bf16", 2, 1, 128, 1, None), ("bf16", 3, 3, 128, 128, None), ("bf16", 7, 1, 64, 129, None), ("f32", 4, 2, 128, 131, [0, 64, 131]),
    ("f32", 2, 1, 64, 1, None),
])
def test_outputs_in_slices_of_wider_tensors(dtype, Hq, Hkv, d, n, cuts, flags):
    """dq, dk and dv side by side in one tensor (as a fused projection takes them), o with a gap behind its rows."""
    dt = DT[dtype][0]
    x = _rows(n, (Hq, Hkv, Hkv, Hq), d, dt, False, n)
    m = 1 if cuts is None else len(cuts) - 1
    with Store(dtype, Hq, Hkv, d, 2 * m, flags=flags) as c:
        first = torch.randn(c.state.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        c.state.copy_(first)
        c.dstate.copy_(first)
        at = torch.arange(2 * m, dtype=torch.int32, device="cuda")
        batch = B.lin_batch(m, None if cuts is None else torch.tensor(cuts, device="cuda"), at[:m], at[m:])
        g2 = _decays("spread", Hkv).cuda()
        dense = [torch.full((n, h, d), 3.0, dtype=dt, device="cuda") for h in (Hq, Hq, Hkv, Hkv)]
        _both(c, x, dense, n, g2, batch)
        state, dstate = c.state.clone(), c.dstate.clone()
        c.state.copy_(first)
        c.dstate.copy_(first)
        wide_o = torch.full((n, Hq + 1, d), 3.0, dtype=dt, device="cuda")
        wide = torch.full((n, Hq + 2 * Hkv + 1, d), 3.0, dtype=dt, device="cuda")
        parts = wide[:, :Hq + 2 * Hkv].split([Hq, Hkv, Hkv], dim=1)
        _both(c, x, [wide_o[:, :Hq], *parts], n, g2, batch)
        for a, b in zip(dense, (wide_o[:, :Hq], *parts)):
            assert torch.equal(a, b)
        assert (wide_o[:, Hq:] == 3.0).all() and (wide[:, -1] == 3.0).all()
        assert torch.equal(state, c.state) and torch.equal(dstate, c.dstate)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 128)])
def test_single_tokens_in_slices(dtype, d):
    dt, Hq, Hkv, n = DT[dtype][0], 10, 2, 5
    q, k, v = _rows(n, (Hq, Hkv, Hkv), d, dt, True, 4)
    slots = torch.tensor([3, -1, 0, 4, 1], dtype=torch.int32, device="cuda")
    with Store(dtype, Hq, Hkv, d, 6, grads=False) as c:
        c.state.copy_(torch.randn(c.state.shape, generator=torch.Generator().manual_seed(2)))
        first = c.state.clone()
        got = []
        for gap in (0, 3):
            c.state.copy_(first)
            wide = torch.full((n, Hq + gap, d), 3.0, dtype=dt, device="cuda")
            B.pkv_lin_attn_step(c.lin, q, k, v, wide[:, :Hq], n, None, slots, torch.cuda.current_stream())
            B.pkv_lin_check(c.lin)
            assert (wide[1] == 3.0).all() and (wide[:, Hq:] == 3.0).all()
            got.append((wide[:, :Hq].clone(), c.state.clone()))
        assert all(torch.equal(a, b) for a, b in zip(*got))
        assert torch.equal(got[0][1][[2, 5]], first[[2, 5]])


@pytest.mark.parametrize("flags", [0, B.PKV_FLAG_LIN_ONE_TERM])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_not_finite_stays_in_its_sequence(d, flags):
    """NaN and infinity in one sequence and in rows of none: the others' bits are those without."""
    Hq, Hkv, n, cuts = 4, 2, 400, [0, 100, 230, 390]
    clean = _rows(n, (Hq, Hkv, Hkv, Hq), d, torch.bfloat16, False, 8)
    g2 = _decays("spread", Hkv).cuda()
    batch_at = torch.tensor(cuts, device="cuda")
    at = torch.arange(6, dtype=torch.int32, device="cuda")
    got = []
    for value in (None, float("nan"), float("inf")):
        x = [t.clone() for t in clean]
        if value is not None:
            for t in x:
                t[150, 0, 5] = value
                t[395] = value
        with Store("bf16", Hq, Hkv, d, 6, flags=flags) as c:
            outs = [torch.zeros_like(t) for t in (x[0], x[0], x[1], x[2])]
            _both(c, x, outs, n, g2, B.lin_batch(3, batch_at, at[:3], at[3:]))
            got.append(outs + [c.state.clone(), c.dstate.clone()])
    for bad in got[1:]:
        for a, b in zip(got[0][:4], bad[:4]):
            assert torch.equal(a[:100], b[:100]) and torch.equal(a[230:], b[230:])
        assert all(torch.equal(got[0][4][s], bad[4][s]) and torch.equal(got[0][5][s - 3], bad[5][s - 3]) for s in (3, 5))
        assert not bad[4][4].isfinite().all() and not bad[0][150:230].isfinite().all()
