"""The benchmark's measured traffic goes with the attention kernel's sources: a
change of them, or of what they include, asks for a new capture, and until then
the benchmark reports none."""
import bench


def test_the_record_is_of_the_present_sources():
    assert bench.measured_traffic() is not None
