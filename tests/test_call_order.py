"""Order of a plan's calls over streams and graph captures, on the CPU: the host
sources, compiled against a model of the runtime (tests/hip_model), with every
launch an operation whose predecessors are known."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if not cxx:
        pytest.skip("no host compiler")
    csrc = os.path.join(ROOT, "all_gather_gemm_agmm_amd", "csrc")
    exe = str(tmp_path_factory.mktemp("model") / "call_order")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I" + os.path.join(HERE, "hip_model"), "-I" + os.path.join(ROOT, "include"),
                    "-I" + csrc, os.path.join(HERE, "call_order_model.cpp"), os.path.join(csrc, "agmm_api.cpp"),
                    os.path.join(csrc, "agmm_ops.cpp"), "-o", exe], check=True)
    return exe


def run_model(exe, *args):
    run = subprocess.run([exe, *args], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and "all in order" in run.stdout, run.stdout + run.stderr


def test_calls_are_ordered(model):
    """Eager calls wait for the last eager call, whatever was captured in
    between; captured calls for the last one of their capture; a plan's end for
    its last eager call."""
    run_model(model)


def test_pieces_that_no_launch_holds_are_refused(model):
    """When they are set, and the plan keeps what it had; accepted ones run."""
    run_model(model, "pieces")
