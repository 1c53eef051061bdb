"""bench.py reports the step kernel's measured DRAM traffic only for the kernel source it was measured on."""
from __future__ import annotations

import bench


def test_the_default_workload_has_traffic_measured_on_this_kernel_source():
    assert ("c4-N108000-H24-d128", bench.kernel_hash()) in bench.NCU_TRAFFIC
