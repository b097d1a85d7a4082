"""A leading token over many small weights: they still count.

The leader's value is zero (what models make of a token that takes the attention which
nobody needs), so the output is the small weights' alone.  Requests share their pages (a
common prefix), so that a warp has hundreds of tokens beside the leader."""
import numpy as np
import pytest

from oracle import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_decode_attention_oasis_gb300 import build

    build.build()


@pytest.mark.parametrize("lead", [176, 192, 224])  # 15.6, 17.0 and 19.8 nats above the others' mean
# a pair to a block of eight warps; equal ranges, several pairs to a warp
@pytest.mark.parametrize("batch,ctx", [(256, 2048), (2500, 1000)])
@pytest.mark.parametrize("at", [0, 70])
def test_small_weights_count(at, batch, ctx, lead):
    from paged_helpers import F16_HALF_STEP, cache_of, check_attention, ints, random_pages

    rng = np.random.default_rng(lead + at)
    n_pages = -(-ctx // 16)
    kv, scale = random_pages(rng, n_pages, 1)
    scale[:] = 2.0 ** -7
    kv[:, 0, 1] &= 0x7f  # values of one sign: their mean is not small against them
    kv[at // 16, 0, 0, at % 16] = ref.e4m3_bytes(np.array(float(lead)))
    kv[at // 16, 0, 1, at % 16] = 0
    table = np.arange(n_pages)[None]
    c = cache_of(kv, scale, np.repeat(table, batch, 0), 2)
    q = torch.ones((batch, 2, 128), dtype=torch.bfloat16, device="cuda")
    got = c.decode(q, ints([ctx] * batch)).double().cpu().numpy()
    want, mass, size, tiny = ref.decode(np.ones((1, 2, 128)), kv, scale, table, [ctx], SCALE)
    # a weight of the largest score is held as 2^11 at least, so half of fp16's smallest step is 2^-36 of it
    check_attention(got, want, mass, size, F16_HALF_STEP, tiny * 2.0 ** -11)


@pytest.mark.parametrize("nb_max", [8, 60, 4000])  # a block to a pair, a cluster, equal ranges
@pytest.mark.parametrize("first", [True, False])
def test_scales_100_binades_apart_share_one_sum(first, nb_max):
    """One page of large values among pages of zeros at the smallest scale: the zeros take their part of the weights."""
    from paged_helpers import F16_HALF_STEP, bf16, cache_of, check_attention, ints, random_pages

    rng = np.random.default_rng(nb_max)
    n_pages = min(nb_max, 300)
    kv, scale = random_pages(rng, n_pages, 1)
    large = 0 if first else n_pages - 1
    scale[:, :, 0] = 2.0 ** -7
    scale[:, :, 1] = 2.0 ** -60
    scale[large, :, 1] = 2.0 ** 40
    kv[np.arange(n_pages) != large, 0, 1] = 0
    table = np.full((1, nb_max), -1)
    table[0, :n_pages] = np.arange(n_pages)
    c = cache_of(kv, scale, table, 3)
    q, q64 = bf16(rng, (1, 3, 128))
    got = c.decode(q, ints([n_pages * 16])).double().cpu().numpy()
    want, mass, size, tiny = ref.decode(q64, kv, scale, table, [n_pages * 16], SCALE)
    check_attention(got, want, mass, size, F16_HALF_STEP, tiny * 2.0 ** -11 / n_pages)  # 16 tokens have values
