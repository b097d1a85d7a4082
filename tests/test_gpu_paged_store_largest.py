"""The largest finite bf16 values pass 448 * 2^119, the largest value of a page: they are stored as that."""
import numpy as np
import pytest

from oracle import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_decode_attention_oasis_gb300 import build

    build.build()


def test_the_largest_finite_values_saturate():
    from paged_helpers import cache_of, ints

    top = torch.finfo(torch.bfloat16).max
    k = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    # 448 * 2^119 itself, the next value of bf16, the largest; 2^109 is half of the smallest step and ties to zero
    k[0, 0, :6] = torch.tensor([1.75 * 2.0 ** 127, 1.7578125 * 2.0 ** 127, top, -top, 2.0 ** 109, 1.5 * 2.0 ** 109])
    kv, scale = np.zeros((1, 1, 2, 16, 128), np.uint8), np.ones((1, 1, 2))
    c = cache_of(kv, scale, np.zeros((1, 1), int), 1)
    c.store(k.cuda(), k.cuda(), ints([0]))
    values = ref.E4M3[c.kv[0, 0, 0, 0, 0].cpu().numpy()] * float(c.scale[0, 0, 0, 0])
    most = 448 * 2.0 ** 119
    assert values[:6].tolist() == [most, most, most, -most, 0.0, 2.0 ** 110]
    assert (values[6:] == 0).all() and np.isfinite(np.float32(most))
    # the error of a finite value is an eighth at most
    assert (top - most) / top < 0.125
