"""Refusals of the permutation and microscaled calls that come after the device check, without a
GPU: tests/c/mx_refusals.cpp stands in for the HIP runtime and counts the launches that a call would
have made."""
import os
import shutil
import subprocess

import pytest

import precision_moe_amd as pm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIP_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE), reason="needs g++ and HIP's headers")
def test_refused_before_the_first_launch(tmp_path):
    exe, lib = tmp_path / "mx_refusals", os.path.dirname(os.path.abspath(pm.LIB_PATH))
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__", "-isystem", HIP_INCLUDE,
                    "-I", os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "mx_refusals.cpp"), "-o", str(exe),
                    "-rdynamic", "-L", lib, "-lpmoe", f"-Wl,-rpath,{lib}"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "refusals: ok" in r.stdout
