"""The DRAM traffic that the benchmark's roofline entry quotes was captured on the
sources that are here."""
import bench

DECODE = ["paged_kv_cache_143_gb300/csrc/" + f
          for f in ("decode.cu", "decode_rows.cuh", "pa_device.cuh")]


def test_traffic_of_the_decode_kernel_is_current():
    assert bench.traffic_for("decode_kernel", DECODE), \
        "the decode kernel's sources changed: take profiles/traffic.json's capture again"


def test_traffic_of_other_sources_is_not_quoted():
    assert bench.traffic_for("decode_kernel", DECODE[:2]) is None
    assert bench.traffic_for("no_such_kernel", DECODE) is None
