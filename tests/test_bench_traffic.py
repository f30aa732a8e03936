"""The memory traffic that bench.py reports is that of the kernels as they are: the committed counter
summaries carry the digest of the current sources."""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_traffic_was_counted_on_these_sources(kernel):
    assert bench.traffic_for(kernel) is not None
