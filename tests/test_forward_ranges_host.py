"""Which K/V tiles the forward kernel's units load and visit, on the host (no GPU): the kernel's own functions, compiled
for the host (forward_ranges.cu)."""
import os
import subprocess

import pytest

from conftest import ROOT

pytest.importorskip("torch")
from variable_length_packed_gb300 import build as vbuild  # noqa: E402


def test_every_tile_of_a_ring_is_visited_and_every_visible_key_is_in_one(tmp_path):
    exe = str(tmp_path / "forward_ranges")
    subprocess.run([vbuild.nvcc(), *vbuild.ARCH, "-std=c++17", "-O2", "--expt-relaxed-constexpr", "-I",
                    os.path.join(ROOT, "include"), "-I", vbuild.CSRC, os.path.join(ROOT, "tests", "forward_ranges.cu"), "-o",
                    exe], check=True, capture_output=True, text=True)
    done = subprocess.run([exe], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
