"""A resumed request's output does not depend on how large a bound its call has."""
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


def _held(bits, ctx, new, hkv, hq, seed):
    """A cache whose requests hold ctx tokens, new rows, their plan."""
    from paged_helpers import bf16, ints, shuffled_table
    from q4_helpers import pages_and_cache

    from sparse_decode_attention_oasis_gb300.paged import Plan

    rng = np.random.default_rng(seed)
    n_pages = sum(-(-n // 16) for n in ctx) + 1
    table = shuffled_table(rng, ctx, max(-(-n // 16) for n in ctx) + 1, n_pages)
    _, c = pages_and_cache(bits, rng, n_pages, hkv, hq, table)
    c.lens.copy_(ints(ctx))
    q, k, v = (bf16(rng, (sum(new), h, 128), 1.5)[0] for h in (hq, hkv, hkv))
    return c, q, k, v, Plan(None, None, ints(np.concatenate([[0], np.cumsum(new)])), None)


# in all 1,024 keys and fewer, more, of one sequence and of several; some that only a cut finishes in time
CASES = [([300], [20]), ([900], [124]), ([900], [125]), ([0], [500]), ([250] * 8, [50] * 8), ([1000, 5], [24, 19]),
         ([1024, 5], [24, 19]), ([3000], [17])]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("ctx,new", CASES)
def test_a_looser_bound_gives_the_same_bits(bits, ctx, new):
    c, q, k, v, plan = _held(bits, ctx, new, 8, 32, sum(ctx) + bits)
    n = sum(new)
    tight = c.resume(q[:n], k[:n], v[:n], plan, sum(ctx))
    for bound in (sum(ctx) + 1, max(sum(ctx), 1000), 1025 + sum(ctx), 40_000):
        assert torch.equal(c.resume(q[:n], k[:n], v[:n], plan, bound), tight), bound
    c.check()


@pytest.mark.parametrize("ctx,new", CASES)
def test_rows_of_keys_behind_the_last_sequence(ctx, new):
    """resume_attn over the same rows in buffers of different lengths."""
    from paged_helpers import ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    c, q, k, v, plan = _held(4, ctx, new, 8, 32, sum(ctx) + 20)
    n, m = sum(new), sum(ctx) + sum(new)
    rows = c.read(m + 1100, new=(k[:n], v[:n], plan.row_start))
    rows.k[m:] = float("nan")
    rows.v[m:] = float("nan")
    err = ints([0])
    tight = resume_attn(q[:n], rows.k[:m], rows.v[:m], plan.row_start, rows.row_start, err=err)
    for keys in (m + 1, m + 200, m + 1100):
        assert torch.equal(resume_attn(q[:n], rows.k[:keys], rows.v[:keys], plan.row_start, rows.row_start, err=err), tight), keys
    assert int(err) == 0


def test_a_graph_with_room_gives_what_tight_calls_give():
    """Captured with room for 2,000 held tokens, replayed at lengths on both sides of 1,024 keys."""
    from paged_helpers import ints

    c, q, k, v, plan = _held(4, [1990], [16], 8, 32, 5)
    q, k, v = q[:16], k[:16], v[:16]
    c.resume(q, k, v, plan, 2000)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.resume(q, k, v, plan, 2000)
    for held in (0, 1, 300, 1007, 1008, 1009, 1990):
        c.lens.copy_(ints([held]))
        g.replay()
        eager = c.resume(q, k, v, plan, held)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), held
    c.check()
