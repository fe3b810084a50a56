"""The HBM traffic that the bench reports beside a kernel comes from a kept profile, and only while the sources it was
measured on are the present ones."""
import bench


def test_decode_traffic_is_of_these_sources():
    assert bench.counter_traffic(bench.GATE_UP_KERNEL, "decode1_gate_up_hbm_traffic.md") == 71091702


def test_prefill_traffic_is_of_these_sources():
    kernel = bench.MFMA_GATE_UP_KERNEL.format(fmt=0)
    traffic = bench.counter_traffic(kernel, "prefill2048_mfma_counters.md")
    assert traffic is not None and abs(traffic / 711202152 - 1) < 1e-3
