"""The DRAM traffic beside the bench's figures (CPU): it comes from the committed captures
of the GEMM kernel, which hold while the sources that they name are what they were.  What
other kernels need is declared elsewhere; a change of the GEMM kernel comes with captures."""
import bench
import pytest


@pytest.mark.parametrize("workload", ["q4b S=9", "a3b S=17", "a3b S=17 fp4", "q4b S=9 sample", "a3b S=17 sample"])
def test_the_captured_traffic_is_that_of_the_current_kernel(workload):
    traffic, source = bench.profiled_traffic(workload)
    assert traffic is not None and traffic > 0, source
