"""The loss's row copy takes as many pieces of 8 columns as its rows have, no
more and no fewer: checked in the built library, where no GPU is visible."""
import os
import shutil
import subprocess

import pytest

import all_gather_gemm_agmm_amd as agmm

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "all_gather_gemm_agmm_amd", "csrc")


def test_piece_counts_that_do_not_fit_are_refused(tmp_path):
    cxx, rocm = shutil.which("g++") or shutil.which("clang++"), os.environ.get("ROCM_PATH", "/opt/rocm")
    if not cxx:
        pytest.skip("no host compiler")
    agmm.load_library()
    exe = str(tmp_path / "row_copy_checks")
    subprocess.run([cxx, "-std=c++17", "-I" + os.path.join(HERE, "hip_model"), "-I" + CSRC,
                    os.path.join(HERE, "row_copy_checks.cpp"), agmm.LIB_PATH, "-Wl,-rpath," + os.path.dirname(agmm.LIB_PATH),
                    "-L" + os.path.join(rocm, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", exe], check=True)
    env = dict(os.environ, HIP_VISIBLE_DEVICES="", ROCR_VISIBLE_DEVICES="")
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60, env=env)
    assert run.returncode == 0 and "all as expected" in run.stdout, run.stdout + run.stderr
