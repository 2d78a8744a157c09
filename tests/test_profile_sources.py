"""A figure that bench.py takes from a stored profile belongs to the sources that were profiled."""
import bench


def test_stored_traffic_belongs_to_the_sources():
    """The GEMM's DRAM bytes a launch: null once its source or the two headers it includes differ from
    those of the capture (a helper that other kernels need goes elsewhere, or the capture is taken again)."""
    assert bench.stored_traffic("umma_gemm.cu", "k_umma_qgemm_up_proj_4096x11008_M4096.md") is not None
