"""The committed profiles' DRAM traffic belongs to the committed kernel
sources, so that the bench line can report it."""
import pytest

import bench


@pytest.mark.parametrize("workload", bench.PROFILES)
def test_traffic_is_of_these_sources(workload):
    name, files = bench.PROFILES[workload]
    assert bench.profiled_traffic(workload) is not None, (
        f"profiles/{name} was captured on other sources: {bench.source_hash(files)}")
