"""Two host threads in the decode attention at once, on a made-up CUDA runtime (no GPU): a call's two
launches stay together, and no thread lowers the shared-memory limit below what another launches with."""
import os
import shutil
import subprocess

import pytest

from sparse_decode_attention_oasis_gb300 import build

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "paged_launch_threads.cpp")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    build.build()
    exe = str(tmp_path_factory.mktemp("paged_launch") / "threads")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    cmd = ["g++", "-std=c++17", "-I", include, SRC, os.path.join(build.OBJ, "paged_attn.o"), "-o", exe, "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def _run(program, mode):
    r = subprocess.run([program, mode], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())


def test_a_calls_launches_are_not_parted(program):
    """The second launch reads what the first one left in the stream's scratch."""
    out = _run(program, "launches")
    assert out["status"] == "0 0"
    order = out["order"]
    assert len(order) == 20 and all(order[i] == order[i + 1] for i in range(0, 20, 2)), order
    assert "ab" in order or "ba" in order  # the threads did meet


def test_limits_of_shared_memory_only_grow(program):
    """A group of one query head needs an eighth of what a group of eight does."""
    assert _run(program, "limits")["status"] == "0 0"
