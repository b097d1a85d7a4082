"""check() sees what was reported on any stream, and a first call may be a captured one."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_decode_attention_oasis_gb300 import build

    build.build()


def test_check_waits_for_other_streams():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.binding import OasisError
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(0)
    c = PagedKV(n_pages=4, batch=1, nb_max=2, n_q_heads=1, n_kv_heads=1)
    k, _ = bf16(rng, (1, 1, 128))
    slots = ints([1000])  # of no page
    c.store(k, k, ints([0]))
    c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # tens of milliseconds
        c.store(k, k, slots)
    with pytest.raises(OasisError, match="BAD_SLOT"):
        c.check()
    torch.cuda.synchronize()
    c.check()  # the word is clear


FIRST = """
import torch
from sparse_decode_attention_oasis_gb300.paged import PagedKV, prompt_attn
c = PagedKV(n_pages=8, batch=2, nb_max={nb_max}, n_q_heads=4, n_kv_heads=1)
c.kv.zero_()
lens = torch.tensor([20, 40], dtype=torch.int32, device="cuda")
q = torch.randn(60, 4, 128, device="cuda").bfloat16()
k = torch.randn(60, 1, 128, device="cuda").bfloat16()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    plan = c.extend(lens, 60)
    a = c.prompt(q, k, k, plan)
    c.store(k, k, plan.slot_map)
    b = c.decode(q[:2], plan.lens)
g.replay()
torch.cuda.synchronize()
c.check()
got = a.clone(), b.clone(), c.kv.clone()
plan = c.extend(lens, 60)
assert torch.equal(c.prompt(q, k, k, plan), got[0])
c.store(k, k, plan.slot_map)
assert torch.equal(c.kv, got[2]) and torch.equal(c.decode(q[:2], plan.lens), got[1])
c.check()
print("same")
"""


@pytest.mark.parametrize("nb_max", [4, 4000])
def test_a_process_whose_first_calls_are_captured(nb_max):
    r = subprocess.run([sys.executable, "-c", FIRST.format(nb_max=nb_max)], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
