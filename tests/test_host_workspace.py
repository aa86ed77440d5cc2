"""The library's workspace caches on the CPU: ``host_workspace.cpp`` compiles
the host API against a CUDA runtime that only logs, and plays host threads and
streams against one another.  Nothing here touches a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_token_dispatch_persistent_gb300", "csrc")


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    exe = str(tmp_path_factory.mktemp("host") / "workspace")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-pthread", "-I", include, "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, "-x", "c++", os.path.join(CSRC, "mk_api.cu"),
                    os.path.join(ROOT, "tests", "host_workspace.cpp"), "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("scenario", ["growth", "growth_ep", "growth_host", "release", "release_host", "per_thread", "recycled_handle",
                                      "captured_call", "captured_call_per_thread", "capture_keeps",
                                      "capture_keeps_ep", "capture_alone", "capture_refused"])
def test_scenario(harness, scenario):
    run = subprocess.run([harness, scenario], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout + run.stderr
