"""Two host threads that share a stream and a workspace, each in a call of another kind, on a made-up CUDA runtime (no
GPU): what a call's first launches leave in the workspace is not overwritten before its last one has read it."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from sparse_decode_attention_oasis_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LAUNCHES = {"resume_kv_q8": 3, "resume_kv_q4": 3, "resume": 2, "decode_q8": 2, "decode_q4": 2}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    build.build()
    exe = str(tmp_path_factory.mktemp("paged_workspace") / "threads")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    objects = sorted(glob.glob(os.path.join(build.OBJ, "paged_*.o"))) + [os.path.join(build.OBJ, "prompt_attn.o")]
    cmd = ["g++", "-std=c++17", "-I", include, "-I", os.path.join(ROOT, "include"),
           os.path.join(ROOT, "tests", "c", "paged_workspace_threads.cpp"), *objects, "-o", exe, "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("first,second", [
    ("resume_kv_q4", "resume"), ("resume", "resume_kv_q8"), ("resume_kv_q8", "resume_kv_q4"), ("resume", "decode_q8"),
    ("resume", "decode_q4"), ("resume_kv_q4", "decode_q4"), ("decode_q4", "resume_kv_q8"), ("decode_q8", "decode_q4")])
def test_launches_of_calls_of_two_kinds_are_not_parted(program, first, second):
    r = subprocess.run([program, first, second], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    out = dict(line.split(" ", 1) for line in r.stdout.strip().splitlines())
    assert out["status"] == "0 0", r.stderr
    order = out["order"]
    assert len(order) == 5 * (LAUNCHES[first] + LAUNCHES[second]), order
    assert re.fullmatch(f"({'a' * LAUNCHES[first]}|{'b' * LAUNCHES[second]})+", order), order
    assert "ab" in order or "ba" in order  # the threads did meet
