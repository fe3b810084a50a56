"""The HBM traffic that the bench reports beside a kernel comes from a kept profile, and only while the sources it was
measured on are the present ones."""
import bench


def test_decode_traffic_is_of_these_sources():
    assert bench.counter_traffic(bench.GATE_UP_KERNEL, "decode1_gate_up_hbm_traffic.md") == 71091702
