"""Plans of the feed-forward block and layer norm on the CPU: their host source,
compiled against a model of the runtime (tests/hip_model), with every launch
recorded instead of run."""
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
    exe = str(tmp_path_factory.mktemp("model") / "feed_plan")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I" + os.path.join(HERE, "hip_model"), "-I" + os.path.join(ROOT, "include"), "-I" + csrc,
                    os.path.join(HERE, "feed_plan_model.cpp"), "-o", exe], check=True)
    return exe


def run_model(exe, part):
    run = subprocess.run([exe, part], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and "all as expected" in run.stdout, run.stdout + run.stderr


def test_calls_run_the_form_they_can_use(model):
    """Whatever is kept, a call launches the form that was priced for it, no
    tiles of 224 where 8 bits of a gated product are kept."""
    run_model(model, "forms")


def test_outputs_at_other_operands_are_refused(model):
    """Every output of every entry point at the address of every other operand,
    but for the pairs that may be in place: refused before anything is launched."""
    run_model(model, "overlaps")
