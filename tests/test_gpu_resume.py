"""Attention of prompts that continue a context against the 64-bit definition."""
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


def _run(past, new, hkv=2, G=4, pad=0, kv_pad=0, scale=SCALE, seed=0, sample=None):
    """Packed rows of sequences with `past` keys before `new` query rows; rows of no sequence hold NaN in the
    inputs and keep what out holds.  sample: how many rows are compared (all by default)."""
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    from sparse_decode_attention_oasis_gb300 import binding as B

    rng = np.random.default_rng(seed)
    q_start = np.concatenate([[0], np.cumsum(new)])
    kv_start = np.concatenate([[0], np.cumsum(np.add(past, new))])
    rows, keys = q_start[-1] + pad, kv_start[-1] + kv_pad
    q, q64 = bf16(rng, (rows, hkv * G, 128), 1.5)
    kv, kv64 = bf16(rng, (keys, 2 * hkv, 128))
    q[q_start[-1]:] = float("nan")
    kv[kv_start[-1]:] = float("nan")
    out = torch.full((rows, hkv * G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = resume_attn(q, kv[:, :hkv], kv[:, hkv:], ints(q_start), ints(kv_start), scale, out, err)
    assert got is out and int(err) == 0
    got = got.double().cpu().numpy()
    assert (got[q_start[-1]:] == 7).all()
    if sample is None:
        want, mass, size, mine, _ = ref.resume(q64[: q_start[-1]], kv64[:, :hkv], kv64[:, hkv:], q_start, kv_start, scale)
        check_attention(got[: q_start[-1]][mine], want[mine], mass[mine], size[mine], BF16_HALF_STEP)
        return
    for i in np.unique(np.concatenate([rng.integers(0, q_start[-1], sample), [0, q_start[-1] - 1]])):
        b = int(np.searchsorted(q_start, i, side="right")) - 1
        last = kv_start[b] + past[b] + i - q_start[b] + 1
        one = ref.resume(q64[i:i + 1], kv64[:, :hkv], kv64[:, hkv:], [0, 1], [kv_start[b], last], scale)
        check_attention(got[i:i + 1], one[0], one[1], one[2], BF16_HALF_STEP)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_group_sizes(G):
    _run([0, 130, 1, 500, 77], [3, 70, 129, 1, 0], G=G, pad=3, kv_pad=5, seed=G)


@pytest.mark.parametrize("past,new", [([0], [1]), ([1], [1]), ([127], [1]), ([128], [1]), ([126], [2]), ([0], [128]), ([1], [128]),
                                      ([255], [2]), ([5000], [1]), ([3000], [17]), ([640], [64]), ([641], [65]), ([0, 0], [0, 1]),
                                      ([100, 0, 0, 50], [0, 30, 0, 1])])
def test_lengths(past, new):
    _run(past, new, seed=sum(past) + sum(new))


def test_without_a_context_it_is_the_prompts_attention():
    _run([0, 0, 0], [200, 1, 77], seed=3)


@pytest.mark.parametrize("count", [31, 32, 33, 100])
def test_many_sequences(count):
    rng = np.random.default_rng(count)
    _run(rng.integers(0, 300, count).tolist(), rng.integers(0, 20, count).tolist(), hkv=1, G=2, seed=count)


@pytest.mark.parametrize("hkv,G,past,new", [(8, 4, [6000], [45]), (1, 1, [40000], [1]), (8, 8, [3000, 10], [700, 300]),
                                            (8, 4, [9000, 0, 64], [1100, 2500, 900]), (2, 3, [20000, 20000], [130, 40])])
def test_work_split_over_the_keys(hkv, G, past, new):
    """Sizes whose items cross the borders of the blocks' ranges."""
    _run(past, new, hkv, G, seed=new[0], sample=40)


@pytest.mark.parametrize("past,new,kv_pad", [([900], [124], 0), ([900], [124], 1), ([0, 300], [700, 24], 0), ([10] * 18, [40] * 18, 0),
                                             ([10] * 20, [40] * 20, 0), ([10] * 20, [40] * 20, 24), ([0], [1024], 0)])
def test_few_keys(past, new, kv_pad):
    """Around 1,024 keys and an item to an SM, up to which no item is cut."""
    _run(past, new, 8, 4, kv_pad=kv_pad, seed=len(new), sample=60)


def test_items_of_more_keys_than_31_bits_count():
    """135,000 new rows: the items of all heads have 2.3e9 keys to read between them."""
    from paged_helpers import BF16_HALF_STEP, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    n, past, hkv, G = 135_000, 1_000, 8, 8
    made = torch.Generator("cuda").manual_seed(9)
    q = torch.randn((n, hkv * G, 128), generator=made, device="cuda", dtype=torch.bfloat16)
    kv = torch.randn((past + n, 2 * hkv, 128), generator=made, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(q, 7.0)
    resume_attn(q, kv[:, :hkv], kv[:, hkv:], ints([0, n]), ints([0, past + n]), out=out)
    assert not (out == 7).all(2).any() and out.isfinite().all()
    rng = np.random.default_rng(9)
    for i in [0, n - 1, *rng.integers(0, n, 14)]:
        h = int(rng.integers(0, hkv))
        one, k, v = (x.double().cpu().numpy() for x in (q[i:i + 1, h * G:h * G + G], kv[: past + i + 1, h:h + 1],
                                                        kv[: past + i + 1, hkv + h:hkv + h + 1]))
        want = ref.resume(one, k, v, [0, 1], [0, past + i + 1], SCALE)
        check_attention(out[i:i + 1, h * G:h * G + G].double().cpu().numpy(), want[0], want[1], want[2], BF16_HALF_STEP)


def test_split_results_are_the_same_every_time():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    rng = np.random.default_rng(4)
    q, _ = bf16(rng, (300, 32, 128))
    kv, _ = bf16(rng, (9300, 16, 128))
    args = (q, kv[:, :8], kv[:, 8:], ints([0, 100, 300]), ints([0, 5100, 9300]))
    first = resume_attn(*args)
    for _ in range(5):
        assert torch.equal(resume_attn(*args), first)


@pytest.mark.parametrize("size", [0.0, 1e-3, 12.0])
def test_query_sizes(size):
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    rng = np.random.default_rng(5)
    q, q64 = bf16(rng, (40, 4, 128), size)
    k, k64 = bf16(rng, (900, 1, 128))
    v, v64 = bf16(rng, (900, 1, 128), 100.0)
    got = resume_attn(q, k, v, ints([0, 40]), ints([0, 900])).double().cpu().numpy()
    want, mass, sizes, _, _ = ref.resume(q64, k64, v64, [0, 40], [0, 900], SCALE)
    check_attention(got, want, mass, sizes, BF16_HALF_STEP)


@pytest.mark.parametrize("past", [100, 4000])
def test_infinities_and_nan_reach_the_rows_that_attend_them(past):
    """In a value of the context: every row.  In a new value: its own row and later ones.  In a query: its row."""
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    rng = np.random.default_rng(6)
    new, hkv, G = 90, 2, 4
    q, _ = bf16(rng, (new, hkv * G, 128))
    k, _ = bf16(rng, (past + new, hkv, 128))
    v, _ = bf16(rng, (past + new, hkv, 128))
    v[30, 0, 5] = float("nan")
    v[past + 41, 1, 9] = float("inf")
    v[past + 60, 1, 9] = float("-inf")
    v[past + 70, 0, 100] = float("nan")
    q[88, 3, 0] = float("inf")
    got = resume_attn(q, k, v, ints([0, new]), ints([0, past + new])).float().cpu()
    odd = torch.zeros((new, hkv * G, 128), dtype=torch.bool)
    odd[:, :G, 5] = odd[41:, G:, 9] = odd[70:, :G, 100] = odd[88, 3] = True
    assert torch.equal(~torch.isfinite(got), odd)
    assert torch.isinf(got[41:60, G:, 9]).all() and torch.isnan(got[60:, G:, 9]).all()


def test_bad_sequences_are_skipped_and_flagged():
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    rng = np.random.default_rng(7)
    q, q64 = bf16(rng, (30, 2, 128))
    kv, kv64 = bf16(rng, (60, 2, 128))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for q_start, kv_start in (([0, 5, 9, 20, 31], [0, 9, 12, 40, 60]),   # too few keys, too many query rows
                              ([-1, 5, 3, 12, 30], [0, 9, 30, 50, 60]),  # outside, decreasing
                              ([0, 10, 20, 25, 30], [0, 20, 10, 30, 61]),
                              ([0, 0, 0, 0, 0], [0, 0, 0, 0, 0])):
        err.zero_()
        out = torch.full((30, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        resume_attn(q, kv[:, :1], kv[:, 1:], ints(q_start), ints(kv_start), out=out, err=err)
        want, mass, size, mine, bits = ref.resume(q64, kv64[:, :1], kv64[:, 1:], q_start, kv_start, SCALE)
        got = out.double().cpu().numpy()
        assert int(err) == bits and (got[~mine] == 7).all()
        check_attention(got[mine], want[mine], mass[mine], size[mine], BF16_HALF_STEP)


def test_captured_replayed_and_beside_another_stream():
    """One graph, replayed with other starts, and eager calls of another size on another stream at the same time."""
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    rng = np.random.default_rng(8)
    q, q64 = bf16(rng, (64, 8, 128))
    kv, kv64 = bf16(rng, (3000, 4, 128))
    q_start, kv_start = ints([0, 64]), ints([0, 3000])
    args = (q, kv[:, :2], kv[:, 2:])
    alone = resume_attn(q[:20], *args[1:], ints([0, 20]), kv_start)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = resume_attn(*args, q_start, kv_start)
    side = torch.cuda.Stream()
    for n, m in ((64, 3000), (1, 2999), (17, 17), (40, 1500)):
        q_start.copy_(ints([0, n]))
        kv_start.copy_(ints([0, m]))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            again = resume_attn(q[:20], *args[1:], ints([0, 20]), ints([0, 3000]))
        torch.cuda.synchronize()
        assert torch.equal(again, alone)
        want, mass, size, mine, _ = ref.resume(q64, kv64[:, :2], kv64[:, 2:], [0, n], [0, m], SCALE)
        check_attention(out.double().cpu().numpy()[mine], want[mine], mass[mine], size[mine], BF16_HALF_STEP)


@pytest.mark.parametrize("bits", [4, 8])
def test_through_the_cache(bits):
    """A serving loop: prompts, continued prompts (one of them new, one alone without new rows), decode steps
    between; each output against the definitions over the pages as they are."""
    from paged_helpers import BF16_HALF_STEP, F16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(bits)
    hkv, G, layers, n_pages = 2, 4, 2, 60
    c = PagedKV(n_pages=n_pages, batch=3, nb_max=20, n_q_heads=hkv * G, n_kv_heads=hkv, layers=layers, bits=bits)
    c.kv.zero_()
    lens = np.zeros(3, int)
    for grow in ([70, 0, 33], [5, 40, 0], [1, 1, 1], [130, 2, 90], [0, 0, 1], [1, 1, 1], [16, 100, 7]):
        total = lens + grow
        rows = int(sum(grow)) + 2
        plan = c.extend(ints(total), rows)
        for layer in range(layers):
            k, k64 = bf16(rng, (rows, hkv, 128))
            v, v64 = bf16(rng, (rows, hkv, 128), 2.0)
            q, q64 = bf16(rng, (rows, hkv * G, 128))
            held = c.read(int(lens.sum()), layer=layer)
            start = plan.row_start.cpu().numpy()
            at = held.row_start.cpu().numpy()
            keys, vals, kv_start = [], [], [0]
            for b in range(3):
                keys += [held.k[at[b]:at[b + 1]].double().cpu().numpy(), k64[start[b]:start[b + 1]]]
                vals += [held.v[at[b]:at[b + 1]].double().cpu().numpy(), v64[start[b]:start[b + 1]]]
                kv_start.append(kv_start[-1] + len(keys[-1]) + len(keys[-2]))
            out = c.resume(q, k, v, plan, int(lens.sum()), layer)
            want, mass, size, mine, _ = ref.resume(q64, np.concatenate(keys), np.concatenate(vals), start, kv_start, SCALE)
            got = out.double().cpu().numpy()
            check_attention(got[mine], want[mine], mass[mine], size[mine], BF16_HALF_STEP)
            assert (got[~mine] == 0).all()
            few = c.resume(q, k, v, plan, int(lens[np.asarray(grow) > 0].sum()), layer)  # the others' tokens need no room
            assert torch.equal(few, out)
            c.store(k, v, plan.slot_map, layer)
            d, d64 = bf16(rng, (3, hkv * G, 128))
            step = c.decode(d, plan.lens, layer).double().cpu().numpy()
            pages = c.kv[layer].cpu().numpy(), c.scale[layer].cpu().numpy()
            if bits == 8:
                want = ref.decode(d64, pages[0], pages[1].astype(np.float64), c.table.cpu().numpy(), total, SCALE)
            else:
                want = ref.decode_q4(d64, *pages, c.table.cpu().numpy(), total, SCALE)
            check_attention(step, want[0], want[1], want[2], F16_HALF_STEP, want[3])
        c.commit(plan)
        lens = total
    c.check()


@pytest.mark.parametrize("bits", [4, 8])
def test_one_call_gives_what_the_two_give(bits):
    """oasis_resume_kv_*, then oasis_read_kv_* and oasis_resume_attn on rows of its own."""
    from paged_helpers import bf16, cache_of, ints, random_pages, shuffled_table
    from q4_helpers import cache_q4, random_pages_q4

    from sparse_decode_attention_oasis_gb300 import binding as B
    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    rng = np.random.default_rng(bits)
    ctx, new = [700, 0, 33, 3000], [5, 90, 0, 17]
    table = shuffled_table(rng, ctx, 200, 300)
    kv, scale = random_pages(rng, 300, 2) if bits == 8 else random_pages_q4(rng, 300, 2)
    c = (cache_of if bits == 8 else cache_q4)(kv, scale, table, 8)
    start, lens = ints(np.concatenate([[0], np.cumsum(new)])), ints(ctx)
    q, _ = bf16(rng, (112, 8, 128), 1.5)
    k, _ = bf16(rng, (112, 2, 128))
    v, _ = bf16(rng, (112, 2, 128))
    out = torch.zeros_like(q)
    n = B.oasis_resume_kv_workspace_bytes(c.shape, 112, 3700)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    call = B.oasis_resume_kv_q8 if bits == 8 else B.oasis_resume_kv_q4
    call(c.shape, q, 1024, k, 256, v, 256, start, 112, c.kv, c.scale, c.table, lens, 3700, SCALE, ws, n, out, 1024, c.err)
    rows = c.read(3812, lens, new=(k, v, start), only_new=True)
    assert torch.equal(out, resume_attn(q, rows.k, rows.v, start, rows.row_start)) and int(c.err) == 0


def test_two_threads_resume_on_one_stream():
    """They share the stream's scratch: read-back, attention and join of a call stay together."""
    import threading

    from paged_helpers import bf16, ints, shuffled_table
    from q4_helpers import cache_q4, random_pages_q4

    from sparse_decode_attention_oasis_gb300.paged import Plan

    rng = np.random.default_rng(1)
    held, calls = [6000, 900, 40], 600
    kv, scale = random_pages_q4(rng, 450, 2)
    c = cache_q4(kv, scale, shuffled_table(rng, held, 400, 450), 8)
    c.lens.copy_(ints(held))
    work = []
    for new in ([3, 40, 0], [0, 7, 200]):
        rows = sum(new)
        q, k, v = (bf16(rng, (rows, h, 128), 1.5)[0] for h in (8, 2, 2))
        work.append((q, k, v, Plan(None, None, ints(np.concatenate([[0], np.cumsum(new)])), None)))
    want = [c.resume(*w, sum(held)).clone() for w in work]
    torch.cuda.synchronize()
    outs, failed, start = [[], []], [], threading.Barrier(2)

    def loop(i):
        try:
            start.wait()
            for _ in range(calls):
                outs[i].append(c.resume(*work[i], sum(held)))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and int(c.err) == 0
    for i in range(2):
        wrong = (torch.stack(outs[i]) != want[i]).flatten(1).any(1).sum()
        assert int(wrong) == 0, f"thread {i}: {int(wrong)} of {calls} outputs differ"


def test_the_scratch_grows_and_is_not_kept_past_its_limit(monkeypatch):
    from paged_helpers import bf16, ints, shuffled_table
    from q4_helpers import cache_q4, random_pages_q4

    from sparse_decode_attention_oasis_gb300 import paged

    rng = np.random.default_rng(2)
    kv, scale = random_pages_q4(rng, 130, 2)
    c = cache_q4(kv, scale, shuffled_table(rng, [2000], 130, 130), 8)
    c.lens.copy_(ints([2000]))
    q, k, v = (bf16(rng, (20, h, 128))[0] for h in (8, 2, 2))
    plan = paged.Plan(None, None, ints([0, 20]), None)
    first = c.resume(q, k, v, plan, 2000)
    (kept,) = c._resume_scratch.values()
    assert torch.equal(c.resume(q, k, v, plan, 3000), first)
    (more,) = c._resume_scratch.values()
    assert more.numel() == kept.numel() + 1000 * 4 * 2 * 128
    assert torch.equal(c.resume(q, k, v, plan, 2000), first)
    monkeypatch.setattr(paged, "_KEPT", 1 << 20)
    assert torch.equal(c.resume(q, k, v, plan, 4000), first)
    (still,) = c._resume_scratch.values()
    assert still is more and int(c.err) == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_the_caches_resume_captured_and_replayed(bits):
    """The whole call in a graph, replayed after the cache has grown, beside an eager call; against the eager call's bits."""
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(20 + bits)
    c = PagedKV(n_pages=300, batch=3, nb_max=100, n_q_heads=16, n_kv_heads=4, bits=bits)
    q, _ = bf16(rng, (40, 16, 128))
    k, _ = bf16(rng, (2000, 4, 128))
    new = ints([20, 0, 20])

    def grow(tokens):
        plan = c.extend(c.lens + ints(tokens), int(sum(tokens)))
        c.store(k[: sum(tokens)], k[-sum(tokens):], plan.slot_map)
        c.commit(plan)

    grow([700, 0, 33])
    plan = c.extend(c.lens + new, 40)
    c.resume(q, k[:40], k[40:80], plan, 1900)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = c.extend(c.lens + new, 40)
        out = c.resume(q, k[:40], k[40:80], captured, 1900)
    for tokens in ([1, 0, 0], [100, 50, 900], [0, 1, 16]):
        grow(tokens)
        eager = c.resume(q, k[:40], k[40:80], c.extend(c.lens + new, 40), 1900)
        g.replay()
        again = c.resume(q, k[:40], k[40:80], captured, 1900)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(again, eager)
    c.check()


def test_a_bound_that_is_too_small_is_reported():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.binding import OasisError
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(9)
    c = PagedKV(n_pages=20, batch=2, nb_max=10, n_q_heads=2, n_kv_heads=1, bits=4)
    plan = c.extend(ints([50, 60]), 110)
    k, _ = bf16(rng, (110, 1, 128))
    c.store(k, k, plan.slot_map)
    c.commit(plan)
    plan = c.extend(ints([53, 62]), 5)
    q, _ = bf16(rng, (5, 2, 128))
    good = c.resume(q, k[:5], k[5:10], plan, 110)
    c.check()
    out = c.resume(q, k[:5], k[5:10], plan, 109)  # the second request does not fit
    assert torch.equal(out[:3], good[:3]) and (out[3:] == 0).all()
    with pytest.raises(OasisError, match="BAD_COUNT"):
        c.check()


def test_refusals():
    from paged_helpers import ints

    from sparse_decode_attention_oasis_gb300.binding import OasisError
    from sparse_decode_attention_oasis_gb300.paged import PagedKV, resume_attn

    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device="cuda")
    k, start, kv_start = q[:, :2], ints([0, 4]), ints([0, 4])
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(v=k[:3]), dict(q_start=start.long()), dict(q_start=start[:1]),
                dict(kv_start=ints([0, 1, 2])), dict(out=q[:3]), dict(err=ints([0, 0])), dict(q=q[0])):
        with pytest.raises(ValueError):
            resume_attn(**{"q": q, "k": k, "v": k, "q_start": start, "kv_start": kv_start, **bad})
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(k=k[:0], v=k[:0]), dict(q=q[:, :7]), dict(k=k[:, :1], v=k[:, :1], q=q.repeat(1, 2, 1))):
        with pytest.raises(OasisError):
            resume_attn(**{"q": q, "k": k, "v": k, "q_start": start, "kv_start": kv_start, **bad})
    c = PagedKV(n_pages=4, batch=1, nb_max=2, n_q_heads=8, n_kv_heads=2)
    plan = c.extend(ints([4]), 4)
    for bad in (dict(n_held=-1), dict(layer=1), dict(q=q[:, :4]), dict(k=q), dict(q=q[:3])):
        with pytest.raises(ValueError):
            c.resume(**{"q": q, "k": k, "v": k, "plan": plan, "n_held": 0, **bad})
