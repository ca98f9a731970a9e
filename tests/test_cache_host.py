"""Parts of the cache attention kernels that the host can run: compiled for it and checked
against models of their own (CPU only)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["cache_ring_check", "cache_cut_check"])
def test_host_checks(tmp_path, name):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / name)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I",
                    os.path.join(ROOT, "conditional_draft_tree_gb300", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "cuda", name + ".cu")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
