"""The benchmark reports the scorer's measured traffic: its record in profiles/ is of the sources as
they are."""

import bench


def test_the_recorded_traffic_is_of_these_sources():
    found = bench.recorded_traffic("score_kernel")
    assert found is not None and found["dram_bytes_per_launch"] > 0
