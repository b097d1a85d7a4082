"""A read-back's row starts are an allocation of their own, whatever mode or call came before."""
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


def _cache():
    from paged_helpers import ints, shuffled_table
    from q4_helpers import cache_q4, random_pages_q4

    rng = np.random.default_rng(0)
    kv, scale = random_pages_q4(rng, 12, 1)
    c = cache_q4(kv, scale, shuffled_table(rng, [70, 0, 40], 6, 12), 2)
    c.lens.copy_(ints([70, 0, 40]))
    return c


def test_after_a_call_in_inference_mode():
    c = _cache()
    with torch.inference_mode():
        inside = c.read(110)
    outside = c.read(110)
    assert inside.row_start.is_inference() and not any(t.is_inference() for t in outside)
    outside.row_start.add_(1)  # in place, outside of the mode
    assert outside.row_start.tolist() == [1, 71, 71, 111] and inside.row_start.tolist() == [0, 70, 70, 110]


def test_after_a_call_outside_of_it():
    c = _cache()
    c.read(110)
    with torch.inference_mode():
        assert all(t.is_inference() for t in c.read(110))


def test_nothing_else_is_kept_or_saved_with_it():
    c = _cache()
    for _ in range(3):
        assert c.read(110).row_start.untyped_storage().nbytes() == 4 * 4


def test_after_a_call_in_a_memory_pool_of_its_own():
    """What a pool's scope allocates does not leave it."""
    c = _cache()
    c.read(110)
    pool = torch.cuda.MemPool()
    with torch.cuda.use_mem_pool(pool):
        inside = c.read(110)
    torch.cuda.synchronize()
    ours = {a["address"] for s in pool.snapshot() for a in s["blocks"] if a["state"] == "active_allocated"}
    assert inside.row_start.data_ptr() in ours
    assert c.read(110).row_start.data_ptr() not in ours
