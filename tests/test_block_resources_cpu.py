"""Register, LDS and scratch budgets of the kernels of the rest of a block, from the
compiler's own report for gfx950: no scratch and no spilled vector registers, and
the workgroups a CU that the launch rules count on.  Compiles the device code
only; no GPU is needed."""
import shutil

import pytest

import test_kernel_resources_cpu as base
from test_layers_resources_cpu import kernels

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not installed")
SOURCES = ["engram_layernorm.hip", "engram_scan.hip", "engram_window.hip", "engram_window_step.hip"]


@pytest.fixture(scope="module")
def resources():
    with pytest.MonkeyPatch.context() as m:
        m.setattr(base, "SOURCES", SOURCES)
        return base._resources()


def test_no_kernel_uses_scratch(resources):
    keys = ("ScratchSize [bytes/lane]", "VGPRs Spill")
    for src in SOURCES:
        assert resources[src]
        for k, r in resources[src].items():
            assert all(r[x] == 0 for x in keys), (k, r)


@pytest.mark.parametrize("src,name,waves,workgroups", [
    ("engram_scan.hip", "scan_kernel", 8, 2),                # chunks on their way beside those that wait
    ("engram_window.hip", "window_fwd_kernel", 4, 2),
    ("engram_window.hip", "window_dq_kernel", 4, 2),
    ("engram_window.hip", "window_dkdv_kernel", 8, 1),
    ("engram_window_step.hip", "window_step_kernel", 4, 2),  # the places that lists are split for
    ("engram_layernorm.hip", "layer_norm_bwd_kernel", 5, 2)])
def test_workgroups_of_a_cu(resources, src, name, waves, workgroups):
    """By LDS (160 KB) and by registers (waves per SIMD times four SIMDs)."""
    for k, r in kernels(resources, src, name).items():
        assert r["LDS Size [bytes/block]"] * workgroups <= 160 * 1024, (k, r)
        assert r["Occupancy [waves/SIMD]"] * 4 >= waves * workgroups, (k, r)
