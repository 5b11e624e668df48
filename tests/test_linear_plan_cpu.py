"""The linear layer's plan on the host: the tiles that the GPU tests say they
reach are those that the plan gives them, and together they are all there are."""
from __future__ import annotations

import os
import subprocess

import pytest

from test_gpu_linear_tiles import BACKWARD, FORWARD

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "memory_bound_engram_amd", "csrc")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "linear_plan")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, "-o", exe,
                    os.path.join(HERE, "linear_plan.cpp")], check=True)

    def of(products):
        text = "\n".join(" ".join(map(str, p)) for p in products)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return of


def kind(tiles):
    return tiles[0], tiles[1] > 0, tiles[2] > 0


def test_tiles_are_those_the_tests_say(plans):
    got = plans([(n, m, k) for n, k, m, _ in FORWARD])
    assert [p[:4] for p in got] == [t for _, _, _, t in FORWARD]
    assert not any(p[4] for p in got)  # none takes the path of few rows
    assert [p[:4] for p in plans([(n, k, m) for n, k, m, _, _ in BACKWARD])] == [t for _, _, _, t, _ in BACKWARD]
    assert [p[:4] for p in plans([(m, k, n) for n, k, m, _, _ in BACKWARD])] == [t for _, _, _, _, t in BACKWARD]


def test_every_kind_of_plan_is_reached():
    large = {(s, whole, cut) for s in range(3) for whole, cut in ((True, False), (False, True), (True, True))}
    small = {(s, whole, cut) for s in (3, 4) for whole, cut in ((True, False), (False, True))}
    for rows in ([t for _, _, _, t in FORWARD], [t for _, _, _, t, _ in BACKWARD], [t for _, _, _, _, t in BACKWARD]):
        assert large | small <= {kind(t) for t in rows}


def test_a_plan_covers_its_product(plans):
    """Whole and cut tiles are all tiles, parts are no more than a quarter of the contraction's stages."""
    sizes = ((256, 256), (128, 128), (128, 128), (64, 128), (32, 128))
    products = [(i, j, c) for i in (1, 31, 32, 33, 64, 65, 257, 4000, 70000) for j in (8, 128, 136, 5120, 131072)
                for c in (1, 8, 64, 72, 4096, 100000)]
    for (i, j, c), (shape, whole, cut, parts, _) in zip(products, plans(products)):
        a, b = sizes[shape]
        assert whole + cut == -(-i // a) * -(-j // b)
        assert parts == 1 if cut == 0 else 1 < parts <= -(-c // 64) // 4, (i, j, c)
