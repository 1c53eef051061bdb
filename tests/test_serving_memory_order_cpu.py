"""Orders between memory accesses that the serving kernels rely on and that no run can show to be
missing: read from the kernels' sources."""
from __future__ import annotations

import os
import re

from temporal_block_sparse_sm_b200 import build as lib_build

KERNELS = ("serving_internal.cuh", "rope_append.cuh", "gqa_rows.cuh", "gqa_tile.cuh")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(lib_build.CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_values_zeroed_in_the_ring_are_ordered_before_the_next_copy():
    """A ring stage is written with ordinary stores (hidden values zeroed) and next by TMA: a proxy fence
    lies between the stores and the arrival that frees the stage."""
    for name, start, end in (("gqa_rows.cuh", "*at = make_uint4(0u, 0u, 0u, 0u);", "mbar_arrive(empty(st))"),
                             ("gqa_tile.cuh", "= make_uint4(0u, 0u, 0u, 0u);", "mbar_arrive(v_ok(st))")):
        text = source(name)
        assert text.count(start) == 1 and text.count(end) == 1
        between = text[text.index(start):text.index(end)]
        assert "fence_proxy_async()" in between or "fence.proxy.async.shared::cta" in between, name


def test_loads_of_what_earlier_kernels_write_are_coherent():
    """The kernels may start while the one in front of them still writes their inputs.  The non-coherent
    path (ld.global.nc, __ldg, __restrict__ const pointers) is for data that nobody writes during a
    kernel's whole life, and its loads may be moved in front of the wait for the earlier kernel."""
    for name in KERNELS:
        text = source(name)
        for form in ("__ldg", "ld.global.nc", "__restrict__", "__ldcv", "__ldlu"):
            assert form not in text, f"{name}: {form}"


def test_tensor_memory_is_taken_after_the_wait_for_earlier_kernels():
    """A block that started early and holds all of an SM's Tensor Memory while it waits for the kernel in
    front would keep that kernel's blocks there from allocating theirs: neither would ever end."""
    text = source("gqa_tile.cuh")
    assert text.count("wait_for_earlier_kernels();") == 1 and text.count("ptx::tmem_alloc(") == 1
    assert text.index("wait_for_earlier_kernels();") < text.index("ptx::tmem_alloc(") < text.index("join_may_start();")
    rows = source("gqa_rows.cuh")
    assert "tmem_alloc" not in rows
