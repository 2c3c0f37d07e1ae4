"""The bench's recorded HBM bytes of the GEMMs are known to be of the sources
that they were counted on; this says whether those are the present ones."""
import bench


def test_traffic_records_are_of_the_present_sources():
    """A change that leaves the GEMMs alone keeps the records: declarations of other operators stay out of the GEMMs'
    sources.  A change of a GEMM needs its bytes counted anew."""
    for name, (_, nbytes) in bench.GATE_UP_TRAFFIC.items():
        assert bench.gate_up_traffic(name) == nbytes
