"""The read-back refuses a kv_start that lies on what its thread blocks read while one of them writes it."""
import ctypes

import numpy as np
import pytest

from sparse_decode_attention_oasis_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


# B = 2, nb_max = 64: lengths at 4096 .. 4103, new starts at 8192 .. 8203, table at 16384 .. 16895
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("start", [4096, 4088, 4100, 8192, 8184, 8200, 16384, 16376, 16640, 16892])
def test_starts_on_the_calls_inputs(lib, bits, start):
    s = binding.PagedShape.of(2, 32, 8, 64, 100)
    call = lib.oasis_read_kv_q4 if bits == 4 else lib.oasis_read_kv_q8
    assert call(ctypes.byref(s), 16, 16, 16384, 4096, 16, 1024, 16, 1024, 8192, 3, 0, start, 32, 32, 5, None, None) == 1
    assert b"kv_start must not overlap" in lib.oasis_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_through_the_cache(bits):
    """The rows' starts of the plan as out's: refused, and nothing is written."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_helpers import ints, shuffled_table
    from q4_helpers import pages_and_cache

    rng = np.random.default_rng(bits)
    values, c = pages_and_cache(bits, rng, 12, 2, 4, shuffled_table(rng, [70, 0, 40], 6, 12))
    c.lens.copy_(ints([70, 0, 40]))
    new = torch.randn((9, 2, 128), device="cuda").to(torch.bfloat16)
    memory = torch.arange(64, dtype=torch.int32, device="cuda")
    start = memory[8:12]
    start.copy_(ints([0, 4, 4, 9]))
    rows = c.read(119, new=(new, new, start))
    assert rows.row_start.tolist() == [0, 74, 74, 119]
    for on in (start, memory[5:9], memory[11:15]):
        before = memory.clone()
        with pytest.raises(binding.OasisError, match="overlap"):
            c.read(119, new=(new, new, start), out=(rows.k, rows.v, on))
        assert torch.equal(memory, before)
    lens = memory[20:23]
    lens.copy_(c.lens)
    with pytest.raises(binding.OasisError, match="overlap"):
        c.read(119, lens, out=(rows.k, rows.v, memory[20:24]))
    for on in (memory[4:8], memory[12:16]):  # beside them
        again = c.read(119, new=(new, new, start), out=(rows.k.clone(), rows.v.clone(), on))
        assert on.tolist() == [0, 74, 74, 119] and torch.equal(again.k, rows.k) and torch.equal(again.v, rows.v)
