"""The recorded HBM traffic belongs to the sources that are there, so that the
benchmark reports it: whoever changes the gate's or GateConv's kernels, or their
launches, takes the counters again."""
from __future__ import annotations

import json
import os

from test_bench_cpu import load_bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_records_are_of_the_current_sources():
    b = load_bench()
    rec = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))
    for k in b.KERNEL_SOURCES:
        assert rec[k]["source_hash"] == b.kernel_source_hash(k), k
        assert b.recorded_traffic(k) == rec[k]["bytes_per_launch"] > 0
    for i, c in enumerate(b.CONFIGS):
        assert b.recorded_config_traffic(i) == rec["configs"][str(i)]["bytes_per_call"] > 0, c
    text = open(os.path.join(ROOT, "profiles", "engram_gate_hbm_traffic_pmc.md")).read()
    for k in b.KERNEL_SOURCES:  # the tables beside them are of the same run
        assert f"{rec[k]['bytes_per_launch']:,}" in text, k
