"""bench.py reports the scan call's measured HBM traffic only while the scan's sources are those that it was measured with.
When they change, even by a line that a kernel does not see, the counters are taken again (the commands are in the profile)
and the profile's source_sha256 with them."""
import bench


def test_the_profile_is_of_these_sources():
    assert bench.measured_traffic() is not None, bench.scan_source_hash()
    # the state-only pass and the full pass read and write at least what the call cannot do without
    assert 762_839_040 <= bench.measured_traffic() < 2 * 762_839_040
