"""The committed DRAM counters belong to the kernels as they are: the bench drops a record whose sources changed."""
import json
from pathlib import Path

import pytest

import bench

RECORDS = sorted((Path(__file__).resolve().parents[1] / "profiles").glob("*.traffic.json"))


@pytest.mark.parametrize("record", RECORDS, ids=lambda f: f.name)
def test_a_record_is_of_the_current_sources(record):
    sources = (bench.PREFILL_SOURCES if "prefill" in record.name else bench.COPY_SOURCES if "copy" in record.name else
               bench.DECODE_SOURCES)
    rec = json.loads(record.read_text())
    assert rec["kernel_source_sha256"] == bench.kernel_source_hash(sources)
    want = int(rec["dram_bytes_per_algorithmic_byte"] * 1.0e8)
    assert bench.traffic_per_launch("", 1.0e8, record.name, sources) == want
