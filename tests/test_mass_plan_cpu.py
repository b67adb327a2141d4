"""The host's choice of how many CTAs share a key tile of mla_attn_mass,
compiled from the library's header: no number of multiprocessors lets a
cluster own two key tiles."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "paged_mla_decode_09_gb300", "csrc")


def test_a_cluster_has_one_key_tile_at_most(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, os.path.join(HERE, "mass_plan_check.cc"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert r.stdout.split() == ["8", "4", "4", "1"]
