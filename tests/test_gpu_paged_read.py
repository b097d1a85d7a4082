"""The cache read back as packed rows: equal to the stored values, in 8 and in 4 bits."""
import numpy as np
import pytest

from oracle import paged_ref as ref

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore")]
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_decode_attention_oasis_gb300 import build

    build.build()


def _compare(rows, want, guard=None):
    """Rows behind the last request's (NaN in want) keep the guard."""
    k, v, start, _ = want
    assert rows.row_start.tolist() == start.tolist()
    for got, w in ((rows.k, k), (rows.v, v)):
        got = got.double().cpu().numpy()
        n = start[-1]
        assert (got[:n] == w[:n]).all()
        if guard is not None:
            assert (got[n:] == guard).all()


def _run(bits, ctx, new=None, hkv=2, pad=0, n_rows=None, seed=0, table=None, only_new=False):
    from paged_helpers import bf16, ints, shuffled_table
    from q4_helpers import pages_and_cache

    rng = np.random.default_rng(seed)
    n_pages = sum(-(-max(n, 0) // 16) for n in ctx) + 2
    if table is None:
        table = shuffled_table(rng, ctx, max(1, max(-(-n // 16) for n in ctx)), n_pages)
    values, c = pages_and_cache(bits, rng, n_pages, hkv, hkv, table)
    fresh = fresh64 = None
    total = sum(max(n, 0) for n in ctx)
    if new is not None:
        start = np.concatenate([[0], np.cumsum(new)])
        wide, wide64 = bf16(rng, (start[-1] + pad, 2 * hkv + 1, 128))
        fresh, fresh64 = (wide[:, :hkv], wide[:, hkv + 1:], ints(start)), (wide64[:, :hkv], wide64[:, hkv + 1:], start)
        total += int(start[-1])
    n_rows = total + 3 if n_rows is None else n_rows
    out = tuple(torch.full((n_rows, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = c.read(n_rows, ints(ctx), new=fresh, out=out, only_new=only_new)
    want = ref.read(values, table, ctx, n_rows, fresh64, only_new)
    _compare(rows, want, 7.0)
    assert rows.k is out[0] and int(c.err) == want[3]
    return c


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hkv", [1, 5, 8])
@pytest.mark.parametrize("ctx,new", [([1], None), ([0], None), ([16, 17, 0, 15], None), ([100], [1]), ([0], [1]), ([0, 0], [0, 0]),
                                     ([33, 0, 16, 1, 700], [5, 40, 0, 16, 1]), ([2500, 3], [0, 900])])
def test_lengths(bits, hkv, ctx, new):
    _run(bits, ctx, new, hkv, pad=2, seed=sum(ctx))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("count", [256, 257, 700])
def test_more_requests_than_threads(bits, count):
    rng = np.random.default_rng(count)
    _run(bits, rng.integers(0, 40, count).tolist(), rng.integers(0, 4, count).tolist())


@pytest.mark.parametrize("bits", [4, 8])
def test_a_long_read(bits):
    """More units than warps at a time."""
    _run(bits, [20000, 0, 9000, 17], [1, 3000, 0, 33], hkv=4)


@pytest.mark.parametrize("n_rows", [0, 1, 39, 40, 41, 59, 60, 89])
def test_requests_that_do_not_fit_get_nothing(n_rows):
    _run(4, [30, 10, 5, 0], [10, 10, 20, 5], n_rows=n_rows)


@pytest.mark.parametrize("bits", [4, 8])
def test_only_requests_with_new_rows(bits):
    _run(bits, [300, 20, 0, 17, 5], [0, 3, 0, 1, 0], only_new=True)
    _run(bits, [300, 20], [0, 0], only_new=True, n_rows=4)
    _run(bits, [300, 20], only_new=True, n_rows=1)
    _run(bits, list(range(600)), [i % 7 // 6 for i in range(600)], hkv=1, only_new=True)


def test_bad_pages_and_lengths():
    table = np.array([[1, 99], [-1, 0]])
    c = _run(8, [20, 32], table=table)
    assert int(c.err) == 2
    c = _run(4, [-5, 20], [3, 0], table=table)
    assert int(c.err) == 2


def test_bad_starts_of_new_rows():
    from paged_helpers import bf16, ints
    from q4_helpers import pages_and_cache

    rng = np.random.default_rng(1)
    values, c = pages_and_cache(4, rng, 4, 1, 1, np.array([[0], [1], [2], [3]]))
    k, k64 = bf16(rng, (10, 1, 128))
    start = [0, 4, 2, 11, 11]
    rows = c.read(100, ints([3, 3, 3, 3]), new=(k, k, ints(start)))
    _compare(rows, ref.read(values, np.array([[0], [1], [2], [3]]), [3] * 4, 100, (k64, k64, start)))
    assert int(c.err) == 8


def test_values_that_are_not_finite():
    """A group of NaN reads back as NaN; a stored infinity as the largest value."""
    from paged_helpers import ints
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    for bits in (4, 8):
        c = PagedKV(n_pages=1, batch=1, nb_max=1, n_q_heads=1, n_kv_heads=1, bits=bits)
        c.table.zero_()
        k = torch.ones((2, 1, 128), dtype=torch.bfloat16, device="cuda")
        k[0, 0, 20], k[1, 0, 3] = float("nan"), float("-inf")
        c.store(k, k, ints([0, 1]))
        got = c.read(2, ints([2])).k[:, 0].float().cpu()
        nan = torch.zeros(2, 128, dtype=torch.bool)
        nan[0, 16:32 if bits == 4 else 17] = bits == 4
        nan[0, 20] = True
        assert torch.equal(torch.isnan(got), nan)
        assert got[1, 3] == (-61440 if bits == 4 else -(1.75 * 2.0 ** 127))


def test_default_lengths_and_layer():
    from paged_helpers import bf16, ints
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(2)
    c = PagedKV(n_pages=8, batch=2, nb_max=4, n_q_heads=4, n_kv_heads=2, layers=2, bits=8)
    plan = c.extend(ints([50, 9]), 59)
    k, _ = bf16(rng, (59, 2, 128))
    c.store(k, -k, plan.slot_map, 1)
    c.commit(plan)
    rows = c.read(59, layer=1)
    assert torch.equal(rows.row_start, plan.row_start) and torch.equal(rows.k, -rows.v)
    assert ((rows.k.float() - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10).all()  # e4m3's half step
    c.check()


def test_captured_and_replayed():
    from paged_helpers import ints
    from q4_helpers import pages_and_cache

    rng = np.random.default_rng(3)
    table = np.arange(40).reshape(2, 20)
    values, c = pages_and_cache(4, rng, 40, 2, 2, table)
    ctx = ints([320, 320])
    c.read(640, ctx)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rows = c.read(640, ctx)
    for n in ([320, 320], [0, 5], [100, 0]):
        ctx.copy_(ints(n))
        g.replay()
        torch.cuda.synchronize()
        _compare(rows, ref.read(values, table, n, 640))


def test_refusals():
    from paged_helpers import ints
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    c = PagedKV(n_pages=2, batch=2, nb_max=2, n_q_heads=2, n_kv_heads=2, bits=4)
    k, start = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda"), ints([0, 1, 3])
    out = torch.zeros((5, 2, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(n_rows=-1), dict(ctx_len=ints([1])), dict(layer=1), dict(new=(k, k[:2], start)), dict(new=(k, k, start[:2])),
                dict(new=(k, k, start.long())), dict(new=(k.float(), k, start)), dict(out=(out, out[:4])), dict(out=(out, out.float())),
                dict(out=(out.transpose(0, 1), out))):
        with pytest.raises(ValueError):
            c.read(**{"n_rows": 5, **bad})


def test_the_rows_of_an_earlier_call_as_out():
    from paged_helpers import ints, shuffled_table
    from q4_helpers import cache_q4, random_pages_q4

    rng = np.random.default_rng(6)
    kv, scale = random_pages_q4(rng, 12, 2)
    c = cache_q4(kv, scale, shuffled_table(rng, [70, 0, 40], 6, 12), 4)
    rows = c.read(120, ints([70, 0, 40]))
    want = c.read(120, ints([33, 0, 17]))
    again = c.read(120, ints([33, 0, 17]), out=rows)
    assert all(x is y for x, y in zip(again, rows))
    assert again.row_start.tolist() == [0, 33, 33, 50] and torch.equal(again.k[:50], want.k[:50]) and torch.equal(again.v[:50], want.v[:50])
    for bad in (rows[:1], (*rows, rows.k), (rows.k, rows.v, rows.row_start[:3]), (rows.k, rows.v, rows.row_start.long())):
        with pytest.raises(ValueError):
            c.read(120, ints([33, 0, 17]), out=bad)


def test_starts_of_many_calls_on_two_streams():
    """Every call's row_start is its own, however many there are."""
    from paged_helpers import ints, shuffled_table
    from q4_helpers import cache_q4, random_pages_q4

    rng = np.random.default_rng(8)
    kv, scale = random_pages_q4(rng, 12, 1)
    c = cache_q4(kv, scale, shuffled_table(rng, [70, 0, 40], 6, 12), 2)
    lens = [(int(rng.integers(0, 71)), 0, int(rng.integers(0, 41))) for _ in range(100)]
    on_gpu = [ints(n) for n in lens]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rows = []
    for i, n in enumerate(on_gpu):
        with torch.cuda.stream(side if i % 3 else torch.cuda.current_stream()):
            rows.append(c.read(110, n))
    torch.cuda.synchronize()
    assert len({r.row_start.data_ptr() for r in rows}) == 100
    for r, (x, _, y) in zip(rows, lens):
        assert r.row_start.tolist() == [0, x, x, x + y] and r.row_start.is_contiguous()
