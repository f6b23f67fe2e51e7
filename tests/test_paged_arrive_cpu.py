"""The counts of a cut tile's parts, compiled for the host: one last part for every tile, whatever the order of arrival,
in the header that every workspace of the library has."""

import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("arrive") / "arrive")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover", "-w", f"-I{CUDA}/include",
                    os.path.join(HERE, "paged_arrive_host.cpp"), "-o", exe], check=True, capture_output=True)
    return exe


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_exactly_one_part_is_the_last(program, seed):
    r = subprocess.run([program, str(seed)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
