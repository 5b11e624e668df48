"""Register and scratch budgets of the layers' kernels, from the compiler's own
report for gfx950: no scratch and no spilled vector registers, and the
workgroups a CU that the launch rules count on.  Compiles the device code only;
no GPU is needed."""
import shutil

import pytest

import test_kernel_resources_cpu as base

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not installed")
SOURCES = ["engram_linear.hip", "engram_qknorm.hip", "engram_decay.hip"]


@pytest.fixture(scope="module")
def resources():
    with pytest.MonkeyPatch.context() as m:
        m.setattr(base, "SOURCES", SOURCES)
        return base._resources()


def kernels(resources, src, name):
    found = {k: r for k, r in resources[src].items() if name in k}
    assert found, name
    return found


def test_no_kernel_uses_scratch(resources):
    keys = ("ScratchSize [bytes/lane]", "VGPRs Spill")
    for src in SOURCES:
        assert resources[src]
        for k, r in resources[src].items():
            assert all(r[x] == 0 for x in keys), (k, r)


def test_linear_tiles(resources):
    """Workgroups to a CU by LDS (160 KB) and registers (waves per SIMD times
    four SIMDs over a workgroup's waves): one of 256 x 256 with 8 waves, two of
    128 x 128 with 4, one of its four-stage form, three of 64 x 128, four of
    32 x 128."""
    tiles = kernels(resources, "engram_linear.hip", "gemm_kernel")
    for shape, waves, workgroups in (("Li256ELi256ELi2ELi4ELi2E", 8, 1), ("Li128ELi128ELi2ELi2ELi2E", 4, 2),
                                     ("Li128ELi128ELi2ELi2ELi4E", 4, 1), ("Li64ELi128ELi1ELi4ELi2E", 4, 3),
                                     ("Li32ELi128ELi1ELi4ELi2E", 4, 4)):
        found = {k: r for k, r in tiles.items() if shape in k}
        assert len(found) == 6, (shape, list(tiles))  # two types; forward, dx and dW
        for k, r in found.items():
            assert r["LDS Size [bytes/block]"] * workgroups <= 160 * 1024, (k, r)
            assert r["Occupancy [waves/SIMD]"] * 4 >= waves * workgroups, (k, r)


def test_decay_walk(resources):
    """Two workgroups of Dc / 16 waves to a CU at heads of 128 x 128, which the
    cut of long sequences into segments counts on."""
    walks = kernels(resources, "engram_decay.hip", "walk_kernel")
    for k, r in walks.items():
        if "Li128ELi128E" not in k:
            continue
        assert r["LDS Size [bytes/block]"] * 2 <= 160 * 1024, (k, r)
        assert r["Occupancy [waves/SIMD]"] * 4 >= 2 * 8, (k, r)
