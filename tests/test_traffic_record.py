"""The DRAM bytes per launch that the bench quotes (profiles/traffic.json) belong to
the kernel sources as they are: after a change to these the GEMVs are captured
again, or the bench has no traffic to report."""
import pytest

import bench


@pytest.mark.parametrize("fmt,bits", [("Q8_0", 8.5), ("Q4_0", 4.5), ("Q4_K", 4.5),
                                      ("Q5_K", 5.5), ("Q6_K", 6.5625)])
def test_traffic_is_of_the_present_sources(fmt, bits):
    got = bench.load_traffic(f"qmv_{fmt}")
    assert got is not None, "sources changed since the capture"
    weights = 4096 * 4096 * bits / 8
    assert weights <= got <= 1.01 * weights + 2 * 4096 * 4
