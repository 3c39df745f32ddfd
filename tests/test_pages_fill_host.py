"""The parities by which the attention kernels fill a query buffer again and, when they leave early, wait for its last copy
(``qe_pages_fill.cuh``), built for the host and followed with simulated barriers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tiered_quantize_evict_gb300", "csrc")


class Barrier:
    """An mbarrier's phases: a wait for a parity passes unless the phase under way has it."""

    def __init__(self):
        self.done = 0

    def passes(self, parity):
        return self.done & 1 != parity


@pytest.fixture(scope="module")
def parities(tmp_path_factory):
    nvcc = next((c for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path_factory.mktemp("fill") / "check")
    subprocess.run([nvcc, "-x", "cu", "-O2", "-std=c++17", "-I", CSRC, os.path.join(ROOT, "tests", "pages_fill_check.cu"), "-o", exe], check=True)
    out = subprocess.run([exe, "9"], capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, x.split())) for x in out.splitlines()]


def test_fills_and_drains(parities):
    for last in range(1, 9):                 # the wait for this buffer's fill number `last` fails
        full, empty = Barrier(), Barrier()
        for n in range(last):
            assert empty.passes(parities[n][0])
            assert not (n and full.done < n)
            if n + 1 < last:
                full.done += 1               # landed, used
                assert not empty.passes(parities[n + 1][0])
                empty.done += 1
        assert not empty.passes(parities[last][0]), "the products of the last copy are not done"
        assert not full.passes(parities[last][1]), "the last copy is under way: leaving has to wait"
        full.done += 1
        assert full.passes(parities[last][1]), "it has landed: leaving waits no longer"


def test_injected_expiry_is_checked():
    import tiered_quantize_evict_gb300 as qe
    if not os.path.exists(qe.LIB_PATH):
        from tiered_quantize_evict_gb300.build import build_library
        build_library()
    for bad in (-1, 1, 3, 7, 2 ** 30 + 1):
        assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, bad) == qe.QE_ERR_INVALID_ARG
    for good in (4, 9, 14, 2 ** 30, 0):
        assert qe.debug_inject(qe.QE_DEBUG_EXPIRE_PAGES_WAIT, good) == qe.QE_OK
