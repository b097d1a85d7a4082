"""The prompt's attention through the cache: its errors reach the cache's check."""
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


def test_errors_are_raised_by_check():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.binding import OasisError
    from sparse_decode_attention_oasis_gb300.paged import PagedKV, prompt_attn

    rng = np.random.default_rng(0)
    c = PagedKV(n_pages=10, batch=2, nb_max=4, n_q_heads=4, n_kv_heads=2)
    q, _ = bf16(rng, (30, 4, 128))
    k, _ = bf16(rng, (30, 2, 128))
    plan = c.extend(ints([20, 10]), 30)
    out = c.prompt(q, k, k, plan)
    assert torch.equal(out, prompt_attn(q, k, k, plan.row_start))
    c.check()
    given = torch.zeros_like(out)
    assert c.prompt(q, k, k, plan, scale=0.3, out=given) is given and not torch.equal(given, out)
    left = c.prompt(q, k, k, plan._replace(row_start=ints([0, 20, 31])))  # the second sequence ends behind the rows
    with pytest.raises(OasisError, match="BAD_COUNT"):
        c.check()
    assert torch.equal(left[:20], out[:20]) and (left[20:] == 0).all()
    c.check()


def test_refusals():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(1)
    c = PagedKV(n_pages=10, batch=2, nb_max=4, n_q_heads=4, n_kv_heads=2)
    q, _ = bf16(rng, (30, 4, 128))
    k, _ = bf16(rng, (30, 2, 128))
    plan = c.extend(ints([20, 10]), 30)
    for bad in (dict(q=q[:, :2]), dict(k=q, v=q), dict(q=q[0]), dict(k=k[0]), dict(v=k[:, :1]), dict(q=q[:5])):
        with pytest.raises(ValueError):
            c.prompt(**{"q": q, "k": k, "v": k, "plan": plan, **bad})
