"""The DRAM traffic that bench.py reports beside the forward sweep was recorded on the
sources that the forward is built from (else it reports none)."""
import bench


def test_recorded_traffic_is_of_the_current_sources():
    assert bench.traffic_for("fwd_sweep") is not None
