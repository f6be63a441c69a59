"""The DRAM traffic that the bench line reports beside a kernel comes from a profiler
capture of these very sources: an edit of one of them without a new capture would
leave the line's figure empty."""
import bench


def test_recorded_traffic_stands_for_the_current_sources():
    for kind in bench.TRAFFIC_SOURCES:
        assert bench.recorded_traffic(kind), kind
