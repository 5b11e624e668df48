"""The recorded kernel times and counters of the rest of a block are of the sources that
are there: whoever changes these kernels takes them again."""
from __future__ import annotations

import hashlib
import os
import re

from test_bench_cpu import load_bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ["engram_device.h", "engram_layers_device.h", "engram_layernorm.hip", "engram_scan.hip", "engram_sequences.h",
           "engram_values.h", "engram_window.hip", "engram_window_bounds.h", "engram_window_step.hip",
           "engram_window_tiles.h"]


def code_hash():
    """Of the sources without their comments."""
    code_only, h = load_bench().code_only, hashlib.sha256()
    for name in SOURCES:
        with open(os.path.join(ROOT, "memory_bound_engram_amd", "csrc", name), encoding="utf-8") as f:
            h.update(code_only(f.read()).encode() + b"\0")
    return h.hexdigest()[:16]


def test_records_are_of_the_current_sources():
    text = open(os.path.join(ROOT, "profiles", "block_kernel_trace.md"), encoding="utf-8").read()
    assert re.search(r"sources (\w{16})", text).group(1) == code_hash()
