"""The bench reports the dominant kernel's DRAM traffic from a committed capture, as long as the
capture was taken on the sources there are."""
import bench


def test_the_traffic_record_is_of_the_present_sources():
    traffic, sha = bench.profile_traffic()
    assert sha is not None
    assert traffic is not None and traffic > 0, "profiles/traffic.json was taken on other sources of the GEMV"
