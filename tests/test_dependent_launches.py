"""Kernels launched as programmatic dependents, read in the source: no row-dependent way out of one lies before its wait.

A dependent launch's wait covers the kernel directly before it, so the order along a chain of such launches holds only if every
grid has itself waited before it completes.  A thread may leave early only where another thread of the same grid, whatever the
data, stays and waits."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_409_b200", "csrc")

# kernel -> ways out before the wait that leave a waiting thread in every grid: beyond the grid's last row, and (the decodes)
# beyond a sequence's last partition, the first of which always stays
ALLOWED = {
    ("decode.cuh", "paged_decode_kernel"): ["part >= nparts"],
    ("decode_mma.cuh", "paged_decode_mma_kernel"): ["part >= nparts"],
    ("decode_fp8.cuh", "paged_decode_fp8_kernel"): ["part >= nparts"],
    ("decode_int8.cuh", "paged_decode_int8_kernel"): ["part >= nparts"],
    ("decode.cuh", "paged_decode_merge_kernel"): ["wid >= p.num_seqs * p.num_q_heads"],
    ("decode_multi.cuh", "paged_decode_multi_merge_kernel"): ["wid >= p.total_q_tokens * p.num_q_heads"],
    ("prefill_int8.cuh", "paged_prefill_int8_kernel"): [],
    ("row_kernels.cuh", "rope_table_kernel"): [],
    ("row_kernels.cuh", "rope_rows_kernel"): [],
    ("row_kernels.cuh", "read_int8_kernel"): [],
}


def body(file, kernel):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    at = src.index("{", re.search(r"\b%s\s*\(" % kernel, src).end())
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i]
    raise AssertionError("no body")


@pytest.mark.parametrize("file,kernel", ALLOWED, ids=lambda x: x if x.endswith("kernel") else "")
def test_nothing_leaves_before_the_wait(file, kernel):
    text = body(file, kernel)
    waits = [m.start() for m in re.finditer(r"(?<!if \(p\.wait_first\) )\bgriddep_wait\(\);", text)]
    assert waits, "the kernel never waits"
    before = text[: waits[0]]
    outs = [m.group(1) for m in re.finditer(r"if \(([^;{}]*)\) return;", before)]
    assert len(outs) == len(re.findall(r"\breturn;", before)), "a return of another form"
    assert outs == ALLOWED[file, kernel]
