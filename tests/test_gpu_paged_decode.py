"""Decode attention over 8-bit pages against the 64-bit definition."""
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


WIDE = 4000  # columns of a table (entries of a selection) beyond which a pair is not left to one cluster


def _inputs(rng, ctx, hkv, hq, q_size=1.0, low=-9, high=-5, wide=False):
    from paged_helpers import bf16, random_pages, shuffled_table

    nb_max = WIDE if wide else max(1, max(-(-n // 16) for n in ctx))
    n_pages = sum(-(-max(n, 0) // 16) for n in ctx) + 3
    kv, scale = random_pages(rng, n_pages, hkv, low, high)
    table = shuffled_table(rng, ctx, nb_max, n_pages)
    used = set(table[table >= 0].tolist())
    for p in range(n_pages):
        if p not in used:
            kv[p] = 0x7f  # pages of nobody hold NaN
    for b, n in enumerate(ctx):
        if n % 16 and n > 0:
            kv[table[b, n // 16], :, :, n % 16:] = 0x7f  # and so do positions behind the last token
    q, q64 = bf16(rng, (len(ctx), hq, 128), q_size)
    return kv, scale, table, q, q64


def _check(c, q, q64, kv, page_scale, table, ctx, sel=None, nsel=None, **kw):
    from paged_helpers import F16_HALF_STEP, check_attention, ints

    out = c.decode(q, ints(ctx), sel=None if sel is None else ints(sel), nsel=None if nsel is None else ints(nsel), **kw)
    want, mass, size, tiny = ref.decode(q64, kv, page_scale, table, ctx, kw.get("scale", SCALE), sel, nsel)
    check_attention(out.double().cpu().numpy(), want, mass, size, F16_HALF_STEP, tiny)
    return out


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_group_sizes(G, wide):
    from paged_helpers import cache_of

    rng = np.random.default_rng(G)
    ctx = [1, 16, 17, 300, 0, 95]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 3, 3 * G, wide=wide)
    c = cache_of(kv, scale, table, 3 * G)
    out = _check(c, q, q64, kv, scale, table, ctx)
    assert (out[4] == 0).all()
    c.check()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ctx", [[1], [15], [0], [0, 0, 5], [31, 32, 33], [4096], [20000, 3], [700] * 9,
                                 list(range(0, 130)), [257, 16, 0, 8000, 1, 2, 0, 0, 500]])
def test_lengths(ctx, wide):
    from paged_helpers import cache_of

    rng = np.random.default_rng(sum(ctx))
    kv, scale, table, q, q64 = _inputs(rng, ctx, 2, 8, wide=wide)
    c = cache_of(kv, scale, table, 8)
    _check(c, q, q64, kv, scale, table, ctx)
    c.check()


def test_many_requests():
    """More pairs than threads of a block: 600 requests of 5 heads, most of them short."""
    from paged_helpers import cache_of

    rng = np.random.default_rng(11)
    ctx = [int(n) for n in rng.integers(0, 40, 600)]
    ctx[17] = 3000
    kv, scale, table, q, q64 = _inputs(rng, ctx, 5, 10)
    c = cache_of(kv, scale, table, 10)
    _check(c, q, q64, kv, scale, table, ctx)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("low,high", [(-60, -59), (-40, 30), (60, 100), (100, 110)])
def test_scales_far_apart(low, high, wide):
    """Scales of neighbouring pages many binades apart, values' above all: the page with the large
    ones decides the output, whatever its weight."""
    from paged_helpers import F16_HALF_STEP, cache_of, check_attention, ints

    rng = np.random.default_rng(high + 100)
    ctx = [200, 33, 1]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 2, 4, low=low, high=high, wide=wide)
    scale[:, :, 0] = 2.0 ** -7  # keys of ordinary size
    c = cache_of(kv, scale, table, 4)
    out = c.decode(q, ints(ctx)).double().cpu().numpy()
    want, mass, size, _ = ref.decode(q64, kv, scale, table, ctx, SCALE)
    # weights are held relative to the largest weight times scale: fp16's 2^-25 is of the largest value's share
    tiny = np.zeros(want.shape[:2] + (1,))
    for b, n in enumerate(ctx):
        for h in range(2):
            tiny[b, 2 * h:2 * h + 2] = n * mass[b, 2 * h:2 * h + 2].max(-1, keepdims=True)
    check_attention(out, want, mass, size, F16_HALF_STEP, tiny)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("q_size", [0.0, 1e-30, 1e-4, 30.0, 1e4])
def test_query_sizes(q_size, wide):
    """From equal weights to a softmax that takes one token; rows of different size in one group."""
    from paged_helpers import cache_of

    rng = np.random.default_rng(12)
    ctx = [500, 70]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 2, 8, q_size=1.0, wide=wide)
    sizes = torch.tensor([q_size, 1.0, q_size, 1e-2, 1.0, q_size, 0.0, 3.0])[:, None]
    q = (q.cpu() * sizes).to(torch.bfloat16)
    c = cache_of(kv, scale, table, 8)
    _check(c, q.cuda(), q.double().numpy(), kv, scale, table, ctx)


@pytest.mark.parametrize("most", [1, 5, 40, 200, WIDE])
def test_selected_blocks(most):
    from paged_helpers import cache_of

    rng = np.random.default_rng(most)
    ctx, hkv = [700, 0, 33, 16, 2000], 4
    kv, scale, table, q, q64 = _inputs(rng, ctx, hkv, 16)
    sel, nsel = np.full((5, hkv, most), -1), np.zeros((5, hkv), int)
    for b, n in enumerate(ctx):
        for h in range(hkv):
            nb = -(-n // 16)
            take = rng.permutation(nb)[: min(most, int(rng.integers(0, nb + 1)))]
            nsel[b, h] = len(take)
            sel[b, h, :len(take)] = take if h % 2 else np.sort(take)  # any order
    c = cache_of(kv, scale, table, 16)
    _check(c, q, q64, kv, scale, table, ctx, sel, nsel)
    c.check()


@pytest.mark.parametrize("wide", [False, True])
def test_bad_entries_are_skipped_and_flagged(wide):
    from paged_helpers import cache_of, ints

    rng = np.random.default_rng(13)
    ctx = [100, 50]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 1, 2, wide=wide)
    table[0, 2], table[1, 0] = kv.shape[0], -1
    c = cache_of(kv, scale, table, 2)
    _check(c, q, q64, kv, scale, table, ctx)
    assert int(c.err) == 2
    c.err.zero_()
    sel, nsel = np.array([[[0, 7, -3, 6]], [[1, 2, 3, 4]]]), np.array([[4], [9]])
    _check(c, q, q64, kv, scale, table, ctx, sel, nsel)
    assert int(c.err) == 1 | 8
    c.err.zero_()
    c.table.fill_(-1)  # nothing left to attend
    assert (c.decode(q, ints(ctx)) == 0).all()
    c.err.zero_()
    _check(c, q, q64, kv, scale, np.full_like(table, -1), [-5, 10 ** 9 if not wide else 500])
    assert int(c.err) == 2


def test_lengths_beyond_the_table_are_clamped():
    from paged_helpers import cache_of

    rng = np.random.default_rng(14)
    kv, scale, table, q, q64 = _inputs(rng, [96, 96], 1, 1)
    c = cache_of(kv, scale, table, 1)
    for beyond in (97, 10 ** 9, 2 ** 31 - 1):
        _check(c, q, q64, kv, scale, table, [beyond, -1])


def test_strided_queries_given_scale_and_output():
    from paged_helpers import bf16, cache_of

    rng = np.random.default_rng(15)
    ctx = [130, 64, 7]
    kv, scale, table, _, _ = _inputs(rng, ctx, 2, 4)
    wide, wide64 = bf16(rng, (3, 9, 128))
    c = cache_of(kv, scale, table, 4)
    out = torch.full((3, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = _check(c, wide[:, 2:6], wide64[:, 2:6], kv, scale, table, ctx, scale=0.31, out=out)
    assert got is out


def test_refusals():
    from paged_helpers import cache_of, ints

    rng = np.random.default_rng(16)
    kv, scale, table, q, _ = _inputs(rng, [40, 40], 2, 4)
    c = cache_of(kv, scale, table, 4)
    ctx = ints([40, 40])
    sel, nsel = ints(np.zeros((2, 2, 3))), ints(np.ones((2, 2)))
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.transpose(1, 2)), dict(ctx_len=ctx.long()), dict(ctx_len=ctx[:1]),
                dict(sel=sel), dict(nsel=nsel), dict(sel=sel[:, :1], nsel=nsel), dict(sel=sel.long(), nsel=nsel),
                dict(layer=1), dict(out=torch.zeros((2, 4, 128), device="cuda"))):
        with pytest.raises(ValueError):
            c.decode(**{"q": q, "ctx_len": ctx, **bad})
    from sparse_decode_attention_oasis_gb300.binding import OasisError

    for s in (0.0, -1.0, float("nan")):
        with pytest.raises(OasisError):
            c.decode(q, ctx, scale=s)


def test_a_long_cache_past_32_bit_offsets():
    """Pages whose byte offset passes 2^32: one request at the end of a pool of 4.3 GB."""
    from paged_helpers import F16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(17)
    n_pages, hkv = 132000, 8
    c = PagedKV(n_pages=n_pages, batch=1, nb_max=4, n_q_heads=8, n_kv_heads=hkv)
    assert c.kv.numel() > 2 ** 32
    pages = [n_pages - 1, 0, n_pages - 2]
    kv = ref.e4m3_bytes(rng.standard_normal((3, hkv, 2, 16, 128)) * 60)
    for i, p in enumerate(pages):
        c.kv[0, p] = torch.from_numpy(kv[i]).cuda()
        c.scale[0, p] = 2.0 ** -7
    c.table[0, :3] = ints(pages)
    k, k64 = bf16(rng, (1, hkv, 128))
    c.store(k, -k, ints([(n_pages - 2) * 16 + 9]))
    kv2, scale2, _ = ref.store(kv, np.full((3, hkv, 2), 2.0 ** -7), k64, -k64, np.array([2 * 16 + 9]))
    q, q64 = bf16(rng, (1, 8, 128))
    out = c.decode(q, ints([42])).double().cpu().numpy()
    want = ref.decode(q64, kv2, scale2, np.array([[0, 1, 2, -1]]), [42], SCALE)
    check_attention(out, want[0], want[1], want[2], F16_HALF_STEP, want[3])


@pytest.mark.parametrize("wide", [False, True])
def test_captured_and_replayed_with_other_lengths(wide):
    from paged_helpers import cache_of, ints

    rng = np.random.default_rng(19)
    kv, scale, table, q, q64 = _inputs(rng, [3000, 3000, 3000], 2, 8, wide=wide)
    kv[kv & 0x7f == 0x7f] = 0
    c = cache_of(kv, scale, table, 8)
    ctx = ints([3000, 1, 0])
    c.decode(q, ctx)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.decode(q, ctx)
    from paged_helpers import F16_HALF_STEP, check_attention

    for n in ([3000, 1, 0], [0, 0, 0], [17, 2999, 1600], [1, 1, 1]):
        ctx.copy_(ints(n))
        g.replay()
        torch.cuda.synchronize()
        want = ref.decode(q64, kv, scale, table, n, SCALE)
        check_attention(out.double().cpu().numpy(), want[0], want[1], want[2], F16_HALF_STEP, want[3])


@pytest.mark.parametrize("wide", [False, True])
def test_two_captured_graphs_and_two_streams(wide):
    """Graphs of two batches replayed at the same time on two streams, and an eager call beside them:
    no call's scratch is another's."""
    from paged_helpers import cache_of, ints

    rng = np.random.default_rng(18)
    cases = []
    for ctx in ([5000, 17, 900], [64, 3000, 1]):
        kv, scale, table, q, q64 = _inputs(rng, ctx, 4, 16, wide=wide)
        cases.append((cache_of(kv, scale, table, 16), q, ints(ctx)))
    eager = [c.decode(q, n).clone() for c, q, n in cases]
    torch.cuda.synchronize()
    graphs = []
    for c, q, n in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.decode(q, n)
        graphs.append((g, out, torch.cuda.Stream()))
    for _ in range(5):
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        again = cases[0][0].decode(cases[0][1], cases[0][2])
        torch.cuda.synchronize()
        assert torch.equal(again, eager[0])
        for (g, out, _), e in zip(graphs, eager):
            assert torch.equal(out, e)
