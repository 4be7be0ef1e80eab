"""Kernels that let the stream's next kernel start while they run, read as source (no GPU).

A kernel allocates all of an SM's tensor memory, and an allocation waits until there is
room. If the next kernel could start before this one has its own, it could be given an SM's
tensor memory first and then wait for this kernel, which would wait for it: without end.
So the next one may be let in only behind the allocation and the CTA's barrier after it, or
where a CTA leaves without allocating."""
import glob
import os
import re

from paged_kv_chunk_chunked_gb300 import build as pkv_build

SIGNAL = re.compile(r"\blaunch_dependents\(\);|griddepcontrol\.launch_dependents;\" :::")


def _kernels(text):
    """(name, body) of each __global__ function."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", text):
        start = at = text.index("{", m.end())
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        yield m.group(1), text[start:at]


def _sources():
    return sorted(glob.glob(os.path.join(os.path.dirname(pkv_build.__file__), "csrc", "*.cu")))


def _good(body):
    """Whether the next kernel is let in only once this one has its tensor memory."""
    body = re.sub(r"if \([^{};]*\) \{[^{}]*\breturn;\s*\}", "", body)     # CTAs that leave early
    alloc = body.find("tmem_alloc(")
    if alloc < 0:
        return True
    barrier = body.find("__syncthreads()", alloc)
    return barrier >= 0 and all(m.start() > barrier for m in SIGNAL.finditer(body))


def test_next_kernel_starts_behind_the_allocation():
    found, bad = [], []
    for path in _sources():
        with open(path) as f:
            for name, body in _kernels(f.read()):
                if SIGNAL.search(body) and "tmem_alloc(" in body:
                    found.append(name)
                    if not _good(body):
                        bad.append(name)
    assert {"lin_part_tc_kernel", "lin_rows_tc_kernel", "lin_cols_tc_kernel"} <= set(found)
    assert not bad


def test_the_reading_itself():
    kernel = "__global__ void x_kernel(int a) { %s }"
    early = "launch_dependents(); if (warp == 1) { tc::tmem_alloc(&b, 512); } __syncthreads();"
    late = "if (!chunk(c)) { launch_dependents(); return; } if (w) { tc::tmem_alloc(&b, 512); } __syncthreads(); launch_dependents();"
    between = "if (w) { tc::tmem_alloc(&b, 512); } launch_dependents(); __syncthreads();"
    assert [_good(b) for s in (early, late, between) for _, b in _kernels(kernel % s)] == [False, True, False]
