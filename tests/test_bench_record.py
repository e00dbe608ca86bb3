"""The DRAM traffic that bench.py reports was measured on the kernels in the tree."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_traffic_record_is_of_these_sources():
    """The record names the digest of the step's kernel sources it was taken with: a change of their
    code has to take it again, or bench.py reports no traffic."""
    import bench
    for workload, record in bench.NS_TRAFFIC.items():
        kernel = {"tile_shape": record["tile_shape"]}
        assert bench.ns_traffic(workload, "bf16", kernel) == record["bytes_per_launch"]
