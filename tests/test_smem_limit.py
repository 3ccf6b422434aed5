"""Kernels' shared-memory limits only grow, whatever the host threads do
(smem_limit of csrc/hisa_kernels.cuh, with a fake runtime)."""
import os
import subprocess

import pytest

from tests.test_abi import ROOT, build_module


def test_a_smaller_limit_does_not_undo_a_larger_one(tmp_path):
    build = build_module()
    if not os.path.exists(build.NVCC):
        pytest.skip("needs nvcc")
    exe = str(tmp_path / "smem_limit_race")
    subprocess.run([build.NVCC, *build.ARCH, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", build.CSRC,
                    os.path.join(ROOT, "tests", "smem_limit_race.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
