"""The bench line's DRAM traffic comes from ncu summaries of the combine's
source; a change to the sources that the combine is compiled from voids them."""
import pytest

import bench


@pytest.mark.parametrize("kind", sorted(bench.TRAFFIC_FILES))
def test_committed_summaries_are_of_the_combine_as_it_is(kind):
    got = bench.recorded_traffic(kind)
    assert got is not None and got["bytes"] > 0 and got["kernel_source_hash"] == bench.kernel_hash()
