"""The work split of the paged attention kernels, compiled for the host: every
unit of work is visited once, and wrong lengths, starts and pages never lead
outside the buffers."""

import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-w", f"-I{CUDA}/include",
                    os.path.join(HERE, "paged_plan_host.cpp"), "-o", exe], check=True, capture_output=True)
    return exe


@pytest.mark.parametrize("seed", [1, 2])
def test_plan_visits_every_unit_once(program, seed):
    r = subprocess.run([program, str(seed)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
