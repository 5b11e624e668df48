"""The bound of the window attention's loads, on the host: whatever is left of a
sequence and however far its rows are apart, every row of a tile that is there can
be read whole, nothing behind the last one, and never the place that stands for
"nothing there"."""
from __future__ import annotations

import os
import subprocess

import pytest

from memory_bound_engram_amd import block, layers

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "memory_bound_engram_amd", "csrc")
BEYOND = 0xF0000000


@pytest.fixture(scope="module")
def bytes_of(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("bounds") / "window_bounds")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, "-o", exe,
                    os.path.join(HERE, "window_bounds.cpp")], check=True)

    def of(rows):
        text = "\n".join(" ".join(map(str, r)) for r in rows)
        return list(map(int, subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()))
    return of


def test_what_is_left_of_a_sequence_never_wraps(bytes_of):
    cases = [(left, most, ld, d)
             for left in (-5, 0, 1, 2, 15, 16, 17, 63, 64, 65, 128, 1950, 2047, 2048, 2049, 32768, 32769, 262144, 262145,
                          299700, block.WINDOW_ROWS_MAX)
             for most in (16, 32, 64)
             for ld in (128, 7168, 8192, 65536, layers.LD_MAX - 8, layers.LD_MAX)
             for d in (8, 72, 128)]
    for (left, most, ld, d), got in zip(cases, bytes_of(cases)):
        rows = max(0, min(left, most))
        assert got == (2 * ((rows - 1) * ld + d) if rows else 0), (left, most, ld, d)
        assert got < BEYOND
        for r in range(rows):  # each row that is there, whole
            assert 2 * (r * ld + d) <= got
