"""Every DRAM traffic figure of profiles/traffic.txt was taken on the kernel source that is there: the
bench reports none for a source that has changed since."""

import pytest

KEYS = ["inv_rope_group_quant_prefill_8k", "wo_a_prefill_8k", "bmm_a8w8_prefill_8k", "rope_kv_insert_prefill_8k"]


@pytest.mark.parametrize("key", KEYS)
def test_captured_traffic_is_of_this_source(key):
    import bench

    value = bench.measured_traffic(key)
    assert value is not None, f"{key}: its source changed after the capture"
    assert value > 1e8
