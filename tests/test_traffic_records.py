"""The DRAM traffic that the benchmark reports beside its roofline comes from captures of the kernel
source as it is: code that only other kernels use stays out of the files that the records name."""
import json
import os

import pytest

import bench

RECORDS = os.path.join(os.path.dirname(os.path.abspath(bench.__file__)), "profiles", "traffic.json")


@pytest.mark.parametrize("workload", ["churn256", "ragged64", "long131k", "decode16"])
def test_records_are_of_the_current_source(workload):
    record = json.load(open(RECORDS))[workload]
    traffic, note = bench.profiled_traffic(workload, bench.kernel_source_hash(),
                                           record["algorithmic_bytes_per_launch"])
    assert traffic == record["dram_bytes_per_launch"], note
