"""The committed counter summaries that bench.py reports from: taken on the
kernel sources as they are.  No GPU needed."""
import bench


def test_page3_traffic_is_reported():
    """bench.py gives a kernel's DRAM traffic from profiles/ only while the
    attention kernels' sources are those it was taken on."""
    assert bench._traffic_from_profiles("attn_bwd_dkdv", "page3") == 17245952
