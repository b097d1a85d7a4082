"""Block tables and slot maps on the GPU against the 64-bit definitions: equal, entry by entry."""
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


def _cache(B, nb_max, n_pages):
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    return PagedKV(n_pages=n_pages, batch=B, nb_max=nb_max, n_q_heads=1, n_kv_heads=1)


def _state(rng, old, nb_max, n_pages):
    """A table whose requests hold `old` tokens in shuffled pages, and the free list of the others."""
    table = np.full((len(old), nb_max), -1)
    order, at = rng.permutation(n_pages), 0
    for b, n in enumerate(old):
        nb = min(-(-max(n, 0) // 16), nb_max)
        table[b, :nb] = order[at:at + nb]
        at += nb
    free = np.full(n_pages, -1)
    free[: n_pages - at] = order[at:]
    return table, free, n_pages - at


def _run(old, new, n_rows, table, free, n_free, n_pages):
    c = _cache(len(old), table.shape[1], n_pages)
    for t, v in ((c.table, table), (c.free, free), (c.lens, old), (c.n_free, [n_free])):
        t.copy_(torch.tensor(np.asarray(v), dtype=torch.int32))
    plan = c.extend(torch.tensor(np.asarray(new), dtype=torch.int32).cuda(), n_rows)
    want = ref.extend_tables(old, new, free, n_free, table, n_rows, n_pages)
    assert (plan.lens.cpu().numpy() == want[0]).all()
    assert int(plan.n_free) == want[1]
    assert (plan.row_start.cpu().numpy() == want[2]).all()
    assert (plan.slot_map.cpu().numpy() == want[3]).all()
    assert (c.table.cpu().numpy() == want[4]).all()
    assert int(c.err) == want[5]
    assert (c.lens.cpu().numpy() == old).all() and int(c.n_free) == n_free  # a plan changes neither
    return c, plan, want


CASES = {
    "one_token": ([0], [1], 1), "nothing": ([0, 7], [0, 7], 3), "one_page": ([0], [16], 16), "page_and_one": ([0], [17], 17),
    "inside_a_page": ([3, 16, 31], [4, 17, 33], 4), "padded": ([0, 40], [20, 41], 50), "no_rows": ([0, 5], [0, 5], 0),
    "rows_short": ([0, 0, 3], [20, 30, 4], 40), "bad_lengths": ([5, -3, 4, 0, 16], [3, 2, 10 ** 6, 9, 17], 12),
}


@pytest.mark.parametrize("name", CASES)
def test_small(name):
    old, new, rows = CASES[name]
    rng = np.random.default_rng(len(name))
    table, free, n = _state(rng, old, 8, 60)
    _run(old, new, rows, table, free, n, 60)


@pytest.mark.parametrize("B,longest,n_pages", [(1, 40000, 3000), (3, 9000, 2000), (256, 200, 4000), (257, 100, 3000),
                                               (700, 70, 4000), (5000, 12, 9000)])
def test_random(B, longest, n_pages):
    rng = np.random.default_rng(B)
    old = rng.integers(0, longest // 2 + 1, B) * (rng.random(B) < 0.6)
    new = old + np.where(rng.random(B) < 0.4, 1, rng.integers(0, longest // 2 + 1, B))
    nb = -(-int(new.max()) // 16) + 1
    table, free, n = _state(rng, old, nb, n_pages)
    _run(old.tolist(), new.tolist(), int((new - old).sum()) + 5, table, free, n, n_pages)


@pytest.mark.parametrize("n_free", [0, 1, 3, 4, 6])
def test_pages_run_out(n_free):
    rng = np.random.default_rng(n_free)
    old, new = [4, 0, 0, 15, 0], [5, 33, 16, 16, 16]  # needs 0, 3, 1, 0, 1
    table, free, _ = _state(rng, old, 4, 30)
    _run(old, new, 80, table, free, n_free, 30)


def test_bad_pages_are_flagged_and_not_used():
    rng = np.random.default_rng(7)
    old, new = [5, 0], [30, 20]
    table, free, n = _state(rng, old, 4, 30)
    free[n - 2] = 30
    free[n - 3] = -7
    table[0, 0] = 999
    _run(old, new, 60, table, free, n, 30)
    table, free, n = _state(rng, old, 4, 30)
    _run(old, new, 60, table, free, 31, 30)  # a free count beyond the list


def test_grow_release_grow():
    rng = np.random.default_rng(9)
    B, n_pages = 40, 600
    c = _cache(B, 20, n_pages)
    lens, table = np.zeros(B, int), c.table.cpu().numpy()
    free, n = c.free.cpu().numpy(), n_pages
    for step in range(6):
        new = np.minimum(lens + rng.integers(0, 90, B), 320)
        plan = c.extend(torch.tensor(new, dtype=torch.int32).cuda(), 5000)
        c.commit(plan)
        lens, n, _, slots, table, _ = ref.extend_tables(lens, new, free, n, table, 5000, n_pages)
        assert (c.table.cpu().numpy() == table).all() and (plan.slot_map.cpu().numpy() == slots).all()
        keep = np.where(rng.random(B) < 0.3, 0, np.where(rng.random(B) < 0.3, lens // 2, lens))
        c.release(torch.tensor(keep, dtype=torch.int32).cuda())
        free, n, _ = ref.release_tables(lens, keep, table, free, n, n_pages)
        lens = keep
        assert (c.lens.cpu().numpy() == lens).all() and int(c.n_free) == n
        assert (c.free.cpu().numpy()[:n] == free[:n]).all()
        held = [table[b, : -(-lens[b] // 16)] for b in range(B)]
        every = np.concatenate(held + [free[:n]])
        assert sorted(every) == list(range(n_pages))  # every page once: held or free
    c.check()


def test_release_refuses_bad_lengths_and_overflow():
    c = _cache(3, 4, 6)
    c.lens.copy_(torch.tensor([20, 5, 64]))
    c.table.copy_(torch.tensor([[0, 1, -1, -1], [9, -1, -1, -1], [2, 3, 4, 5]]))
    c.n_free.fill_(3)
    free = c.free.cpu().numpy()
    want = ref.release_tables([20, 5, 64], [21, 0, 16], c.table.cpu().numpy(), free, 3, 6)
    c.release(torch.tensor([21, 0, 16], dtype=torch.int32).cuda())
    assert (c.free.cpu().numpy() == want[0]).all() and int(c.n_free) == want[1] and int(c.err) == want[2] == 1 | 4 | 8
    assert c.lens.tolist() == [20, 0, 16]
    with pytest.raises(Exception, match="BAD_BLOCK"):
        c.check()
    c.check()


def test_captured_step_replays():
    c = _cache(4, 8, 40)
    new = torch.zeros(4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.extend(new, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan = c.extend(c.lens + 1, 4)
        c.commit(plan)
    old, table, free, n = np.zeros(4, int), c.table.cpu().numpy(), c.free.cpu().numpy(), 40
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        old, n, start, slots, table, _ = ref.extend_tables(old, old + 1, free, n, table, 4, 40)
        assert (plan.slot_map.cpu().numpy() == slots).all() and (c.table.cpu().numpy() == table).all()
        assert (c.lens.cpu().numpy() == old).all() and int(c.n_free) == n
