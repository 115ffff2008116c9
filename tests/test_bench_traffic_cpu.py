"""The DRAM traffic that the benchmark reports was measured on the kernel source as it is."""
import bench


def test_the_measured_traffic_describes_the_committed_kernel():
    assert bench.measured_traffic() == bench.TRAFFIC_BYTES
    # the floor of the workload's gathered rows, and no more than a third above it
    assert 42.4e6 < bench.TRAFFIC_BYTES < 1.33 * 42.5e6
