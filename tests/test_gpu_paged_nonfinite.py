"""Query rows that hold NaN or infinity: the row's output is NaN as the definition's is, however its
pages were split, and no other row knows of it."""
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


# contexts, columns of the table: one page of one warp; a pair by one block; by a cluster of blocks; by equal
# ranges, where long pairs cross blocks
SPLITS = {"page": ([5, 16, 0], 4), "block": ([100, 70, 0], 8), "cluster": ([900, 333, 0], 60), "ranges": ([9000, 4100, 0], 4000)}


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("split", SPLITS)
def test_one_row_of_a_group(split, value):
    from paged_helpers import F16_HALF_STEP, bf16, cache_of, check_attention, ints, random_pages, shuffled_table

    ctx, nb_max = SPLITS[split]
    rng = np.random.default_rng(len(split))
    n_pages, hkv, hq = sum(-(-n // 16) for n in ctx), 2, 8
    kv, scale = random_pages(rng, n_pages, hkv)
    table = shuffled_table(rng, ctx, nb_max, n_pages)
    q, q64 = bf16(rng, (3, hq, 128))
    c = cache_of(kv, scale, table, hq)
    bad = q.clone()
    for b, h, d in ((0, 1, 17), (0, 6, 0), (1, 4, 127), (2, 3, 5)):
        bad[b, h, d] = value
    got = c.decode(bad, ints(ctx)).double().cpu().numpy()
    want = ref.decode(q64, kv, scale, table, ctx, SCALE)
    assert (got[2] == 0).all()  # no token: zero, whatever the query holds
    hit = np.zeros((3, hq), bool)
    hit[[0, 0, 1], [1, 6, 4]] = True
    assert np.isnan(got[hit]).all()
    for b in range(2):
        ok = ~hit[b]
        check_attention(got[b, ok], want[0][b, ok], want[1][b, ok], want[2][b, ok], F16_HALF_STEP, want[3][b, ok])


@pytest.mark.parametrize("split", ["block", "cluster", "ranges"])
def test_scores_of_minus_infinity_have_no_weight(split):
    """An infinity in the query meets keys of the other sign first, and one finite score is left: the
    tokens before it, -inf, weigh nothing.  With no finite score at all the row is NaN (0 / 0)."""
    from paged_helpers import bf16, cache_of, ints, shuffled_table

    ctx, nb_max = SPLITS[split]
    rng = np.random.default_rng(5)
    n_pages = sum(-(-n // 16) for n in ctx)
    kv = ref.e4m3_bytes(-np.ones((n_pages, 1, 2, 16, 128)))
    scale = np.ones((n_pages, 1, 2))
    table = shuffled_table(rng, ctx, nb_max, n_pages)
    c = cache_of(kv, scale, table, 1)
    q, _ = bf16(rng, (3, 1, 128))
    q[:] = 0
    q[:, 0, 9] = 3e38
    # 3e38 * -1 * 2^119 passes the largest fp32: -inf
    c.scale[0, :, :, 0] = 2.0 ** 119
    assert torch.isnan(c.decode(q, ints(ctx))[:2]).all()
    page = int(table[0, -(-ctx[0] // 16) - 1])  # its first token's score is 0, the others' are finite and lower
    c.scale[0, page, 0, 0] = 1.0
    c.kv[0, page, 0, 0, 0] = 0
    c.kv[0, page, 0, 1] = int(ref.e4m3_bytes(np.array(2.0)))
    out = c.decode(q, ints(ctx))
    assert (out[0] == 2).all() and torch.isnan(out[1]).all()
