"""The distance bias with slopes on every side of what the kernels distinguish:
none, gentle and steep ones (the tensor-core forward bounds the maximum of a
tile while slope * 127 * log2 e <= 64, 0.349, and forms it above that), negative
ones. Bounds are mod_oracle's."""
import pytest
import torch

from paged_kv_chunk_chunked_gb300 import binding as B
from paged_kv_chunk_chunked_gb300 import build as pkv_build
from test_gpu_attn_mod import Case

pytestmark = pytest.mark.gpu

SLOPES = [0.0, 0.34, 0.36, 0.92, 4.0, -0.01, -0.36, 2.0 ** -8]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pkv_build.build()
    B.lib()
    torch.cuda.set_device(0)


def _check(c):
    c.slopes = torch.tensor(SLOPES[:c.Hq])
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    c.mod = B.score_mod(c.cap, c.slopes.cuda(), dev(c.k_begin), dev(c.k_end))
    c.check()


@pytest.mark.parametrize("mask", ["causal", "docs", "prefix", "future"])
@pytest.mark.parametrize("d,Hkv", [(64, 2), (128, 4)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_tensor_core_chunks(d, Hkv, cap, mask):
    _check(Case("bf16", 8, Hkv, d, 128, 700, 200, extra=60, cap=cap, mask=mask, seed=41))


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("mask", ["causal", "window", "future"])
def test_few_queries(n, mask):
    _check(Case("bf16", 8, 2, 64, 128, 900, n, extra=50, mask=mask, seed=42))


@pytest.mark.parametrize("dtype,P", [("f32", 16), ("bf16", 32)])
@pytest.mark.parametrize("mask", ["causal", "future"])
def test_cuda_core_chunks(dtype, P, mask):
    _check(Case(dtype, 8, 4, 64, P, 200, 60, extra=50, mask=mask, seed=43))
