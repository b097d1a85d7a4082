"""No bit of a row's output depends on rows that are not its sequence's: padding, and other sequences' queries, which lie
in the same tiles of 128 rows."""
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


def _inputs(rng, past, new, hkv, G):
    """Rows of sequences with `past` keys before `new` query rows, 64 rows behind them; their starts."""
    from paged_helpers import bf16, ints

    q_start = np.concatenate([[0], np.cumsum(new)])
    kv_start = np.concatenate([[0], np.cumsum(np.add(past, new))])
    q, _ = bf16(rng, (q_start[-1] + 64, hkv * G, 128), 1.5)
    kv, _ = bf16(rng, (kv_start[-1], 2 * hkv, 128), 1.5)
    return q, kv[:, :hkv], kv[:, hkv:], ints(q_start), ints(kv_start)


def _others(q, n):
    """What rows n .. may hold instead."""
    yield torch.zeros_like(q[n:])
    yield q[n:] * 30
    yield torch.full_like(q[n:], float("nan"))
    yield torch.full_like(q[n:], float("inf"))
    yield torch.full_like(q[n:], 3e38)


@pytest.mark.parametrize("past,new,hkv,G", [([3000], [17], 8, 4), ([900], [124], 8, 4), ([250] * 8, [50] * 8, 8, 4),
                                            ([5000, 40], [70, 3], 2, 3), ([0], [600], 1, 8), ([700, 0], [1, 129], 2, 5)])
def test_padding_of_a_resumed_prompt(past, new, hkv, G):
    from paged_helpers import ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    q, k, v, q_start, kv_start = _inputs(np.random.default_rng(sum(past) + G), past, new, hkv, G)
    n, err = sum(new), ints([0])
    tight = resume_attn(q[:n], k, v, q_start, kv_start, err=err)
    for rows in (n + 1, n + 64):
        assert torch.equal(resume_attn(q[:rows], k, v, q_start, kv_start, err=err)[:n], tight)
    for other in _others(q, n):
        got = resume_attn(torch.cat([q[:n], other]), k, v, q_start, kv_start, err=err)
        assert torch.equal(got[:n], tight) and (got[n:] == 0).all()
    assert int(err) == 0


@pytest.mark.parametrize("lens,hkv,G", [([17], 8, 4), ([300, 40], 2, 4), ([129, 1, 600], 1, 8), ([1000], 2, 3), ([50] * 12, 2, 2)])
def test_padding_of_prompts(lens, hkv, G):
    from paged_helpers import ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    q, k, v, start, _ = _inputs(np.random.default_rng(sum(lens) + G), [0] * len(lens), lens, hkv, G)
    n, err = sum(lens), ints([0])
    tight = prompt_attn(q[:n], k, v, start, err=err)
    behind = torch.zeros_like(k[:1]).expand(64, -1, -1)
    k, v = torch.cat([k, behind]), torch.cat([v, behind])
    for other in [q[n:], *_others(q, n)]:
        got = prompt_attn(torch.cat([q[:n], other]), k, v, start, err=err)
        assert torch.equal(got[:n], tight) and (got[n:] == 0).all()
    assert int(err) == 0


@pytest.mark.parametrize("past", [0, 800])
def test_queries_of_the_next_sequence(past):
    """They follow in the first one's last tile."""
    from sparse_decode_attention_oasis_gb300.paged import prompt_attn, resume_attn

    new, G = [300, 60], 4
    q, k, v, q_start, kv_start = _inputs(np.random.default_rng(past), [past] * 2, new, 2, G)
    q = q[: sum(new)]

    def run(q):
        return resume_attn(q, k, v, q_start, kv_start) if past else prompt_attn(q, k, v, q_start)

    first = run(q)[: new[0]]
    for other in _others(q, new[0]):
        assert torch.equal(run(torch.cat([q[: new[0]], other]))[: new[0]], first)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("ctx,new", [([300], [20]), ([900], [124]), ([0], [500]), ([250] * 8, [50] * 8), ([1000, 5], [24, 19]),
                                     ([3000], [17])])
def test_padding_of_the_caches_resume(bits, ctx, new):
    from paged_helpers import bf16, ints, shuffled_table
    from q4_helpers import pages_and_cache

    from sparse_decode_attention_oasis_gb300.paged import Plan

    rng = np.random.default_rng(sum(ctx) + 10 + bits)
    n_pages = sum(-(-n // 16) for n in ctx) + 1
    _, c = pages_and_cache(bits, rng, n_pages, 8, 32, shuffled_table(rng, ctx, max(-(-n // 16) for n in ctx) + 1, n_pages))
    c.lens.copy_(ints(ctx))
    n = sum(new)
    q, k, v = (bf16(rng, (n + 64, h, 128), 1.5)[0] for h in (32, 8, 8))
    plan = Plan(None, None, ints(np.concatenate([[0], np.cumsum(new)])), None)
    tight = c.resume(q[:n], k[:n], v[:n], plan, sum(ctx))
    for rows in (n + 1, n + 64):
        out = torch.full_like(q[:rows], 7.0)
        c.resume(q[:rows], k[:rows], v[:rows], plan, sum(ctx), out=out)
        assert torch.equal(out[:n], tight) and (out[n:] == 7).all()
    c.check()
