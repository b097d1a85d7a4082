"""Decode attention over 4-bit pages against the 64-bit definition."""
import numpy as np
import pytest

from oracle import paged_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
SCALE = 128 ** -0.5
WIDE = 6000  # columns of a table beyond which a pair is not left to one cluster


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_decode_attention_oasis_gb300 import build

    build.build()


def _inputs(rng, ctx, hkv, hq, low=12, high=14, wide=False):
    from paged_helpers import bf16, shuffled_table
    from q4_helpers import random_pages_q4

    nb_max = WIDE if wide else max(1, max(-(-n // 16) for n in ctx))
    n_pages = sum(-(-max(n, 0) // 16) for n in ctx) + 3
    kv, scale = random_pages_q4(rng, n_pages, hkv, low, high)
    table = shuffled_table(rng, ctx, nb_max, n_pages)
    used = set(table[table >= 0].tolist())
    for p in range(n_pages):
        if p not in used:
            scale[p] = ref.S_NAN  # pages of nobody hold NaN
    for b, n in enumerate(ctx):
        if n % 16 and n > 0:  # and so do positions behind the last token
            p = table[b, n // 16]
            scale[p, :, 0].reshape(hkv, 16, 8)[:, n % 16:] = ref.S_NAN
            scale[p, :, 1].reshape(hkv, 8, 16)[:, :, n % 16:] = ref.S_NAN
    q, q64 = bf16(rng, (len(ctx), hq, 128))
    return kv, scale, table, q, q64


def _check(c, q, q64, kv, page_scale, table, ctx, sel=None, nsel=None, **kw):
    from paged_helpers import F16_HALF_STEP, check_attention, ints

    out = c.decode(q, ints(ctx), sel=None if sel is None else ints(sel), nsel=None if nsel is None else ints(nsel), **kw)
    want, mass, size, tiny = ref.decode_q4(q64, kv, page_scale, table, ctx, kw.get("scale", SCALE), sel, nsel)
    check_attention(out.double().cpu().numpy(), want, mass, size, F16_HALF_STEP, tiny)
    return out


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_group_sizes(G, wide):
    from q4_helpers import cache_q4

    rng = np.random.default_rng(G)
    ctx = [1, 16, 17, 300, 0, 95]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 3, 3 * G, wide=wide)
    c = cache_q4(kv, scale, table, 3 * G)
    out = _check(c, q, q64, kv, scale, table, ctx)
    assert (out[4] == 0).all()
    c.check()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ctx", [[1], [15], [0], [0, 0, 5], [31, 32, 33], [4096], [20000, 3], [700] * 9,
                                 list(range(0, 130)), [257, 16, 0, 8000, 1, 2, 0, 0, 500]])
def test_lengths(ctx, wide):
    from q4_helpers import cache_q4

    rng = np.random.default_rng(sum(ctx))
    kv, scale, table, q, q64 = _inputs(rng, ctx, 2, 8, wide=wide)
    c = cache_q4(kv, scale, table, 8)
    _check(c, q, q64, kv, scale, table, ctx)
    c.check()


def test_many_requests():
    from q4_helpers import cache_q4

    rng = np.random.default_rng(11)
    ctx = [int(n) for n in rng.integers(0, 40, 600)]
    ctx[17] = 3000
    kv, scale, table, q, q64 = _inputs(rng, ctx, 5, 10)
    c = cache_q4(kv, scale, table, 10)
    _check(c, q, q64, kv, scale, table, ctx)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("low,high", [(0, 2), (4, 14), (20, 27)])
def test_scales_from_the_least_to_the_largest(low, high, wide):
    """Value scales over the whole range, keys of ordinary size."""
    from q4_helpers import cache_q4

    rng = np.random.default_rng(high)
    ctx = [200, 33, 1]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 2, 4, low=low, high=high, wide=wide)
    used = scale[:, :, 0] != ref.S_NAN
    scale[:, :, 0][used] = 100
    c = cache_q4(kv, scale, table, 4)
    _check(c, q, q64, kv, scale, table, ctx)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-4, 30.0])
def test_query_sizes_and_large_keys(size):
    from q4_helpers import cache_q4

    rng = np.random.default_rng(12)
    ctx = [500, 70]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 2, 8)
    sizes = torch.tensor([size, 1.0, size, 1e-2, 1.0, size, 0.0, 3.0])[:, None]
    q = (q.cpu() * sizes).to(torch.bfloat16)
    c = cache_q4(kv, scale, table, 8)
    _check(c, q.cuda(), q.double().numpy(), kv, scale, table, ctx)


@pytest.mark.parametrize("most", [1, 5, 40, 200, WIDE])
def test_selected_blocks(most):
    from q4_helpers import cache_q4

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
    c = cache_q4(kv, scale, table, 16)
    _check(c, q, q64, kv, scale, table, ctx, sel, nsel)
    c.check()


def test_bad_entries_are_skipped_and_flagged():
    from paged_helpers import ints
    from q4_helpers import cache_q4

    rng = np.random.default_rng(13)
    ctx = [100, 50]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 1, 2)
    table[0, 2], table[1, 0] = kv.shape[0], -1
    c = cache_q4(kv, scale, table, 2)
    _check(c, q, q64, kv, scale, table, ctx)
    assert int(c.err) == 2
    c.err.zero_()
    _check(c, q, q64, kv, scale, table, ctx, np.array([[[0, 7, -3, 6]], [[1, 2, 3, 4]]]), np.array([[4], [9]]))
    assert int(c.err) == 1 | 8
    c.table.fill_(-1)
    assert (c.decode(q, ints(ctx)) == 0).all()


def test_nan_stays_where_it_is():
    """A value group of NaN: its 16 dimensions in the rows of its request and head.  A key group of NaN: all of
    those rows.  A query row of NaN: itself."""
    from paged_helpers import ints
    from q4_helpers import cache_q4

    rng = np.random.default_rng(14)
    ctx = [90, 40, 333]
    kv, scale, table, q, _ = _inputs(rng, ctx, 2, 4)
    scale[table[0, 3], 1, 1].reshape(8, 16)[5, 7] = ref.S_NAN
    scale[table[1, 1], 0, 0].reshape(16, 8)[2, 6] = ref.S_NAN
    q[2, 1, 70] = float("nan")
    out = cache_q4(kv, scale, table, 4).decode(q, ints(ctx)).float().cpu()
    want = torch.zeros((3, 4, 128), dtype=torch.bool)
    want[0, 2:, 80:96] = want[1, :2] = want[2, 1] = True
    assert torch.equal(torch.isnan(out), want) and not torch.isinf(out).any()


def test_a_leading_token_with_a_zero_value():
    """One token takes nearly the whole softmax and its value is zero: the others' small weights are the output."""
    from paged_helpers import F16_HALF_STEP, check_attention, ints
    from q4_helpers import cache_q4

    rng = np.random.default_rng(15)
    ctx = [64]
    kv, scale, table, q, q64 = _inputs(rng, ctx, 1, 1)
    p = table[0, 1]
    kv[p, 0, 0, 4] = np.where(q64[0, 0, ::2] > 0, 6, 14) | np.where(q64[0, 0, 1::2] > 0, 6, 14) << 4
    scale[p, 0, 0].reshape(16, 8)[4] = 112  # 4 * 0.5 along the query's signs: some 17 nats ahead
    kv[p, 0, 1, 4] = 0
    c = cache_q4(kv, scale, table, 1)
    out = c.decode(q, ints(ctx)).double().cpu().numpy()
    want, mass, size, tiny = ref.decode_q4(q64, kv, scale, table, ctx, SCALE)
    # a weight below 2^-25 of the largest is off by 2^-36 of that one: `tiny` counts 2^-25 of it
    check_attention(out, want, mass, size, F16_HALF_STEP, tiny * 2.0 ** -11)


def test_strided_queries_given_scale_output_and_layer():
    from paged_helpers import bf16
    from q4_helpers import cache_q4
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(16)
    ctx = [130, 64, 7]
    kv, scale, table, _, _ = _inputs(rng, ctx, 2, 4)
    wide, wide64 = bf16(rng, (3, 9, 128))
    one = cache_q4(kv, scale, table, 4)
    c = PagedKV(n_pages=kv.shape[0], batch=3, nb_max=table.shape[1], n_q_heads=4, n_kv_heads=2, layers=3, bits=4)
    c.kv[2], c.scale[2] = one.kv[0], one.scale[0]
    c.adopt(table=one.table)
    out = torch.full((3, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = _check(c, wide[:, 2:6], wide64[:, 2:6], kv, scale, table, ctx, scale=0.31, out=out, layer=2)
    assert got is out


def test_a_long_cache_past_32_bit_offsets():
    """Pages whose byte offset passes 2^32: requests at the end of a pool of 4.3 GB, written, attended and read back."""
    from paged_helpers import F16_HALF_STEP, bf16, check_attention, ints
    from q4_helpers import random_pages_q4
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(17)
    n_pages, hkv = 264000, 8
    c = PagedKV(n_pages=n_pages, batch=1, nb_max=4, n_q_heads=8, n_kv_heads=hkv, bits=4)
    assert c.kv.numel() > 2 ** 32
    pages = [n_pages - 1, 0, n_pages - 2]
    kv, scale = random_pages_q4(rng, 3, hkv)
    for i, p in enumerate(pages):
        c.kv[0, p], c.scale[0, p] = torch.from_numpy(kv[i]).cuda(), torch.from_numpy(scale[i]).cuda()
    c.table[0, :3] = ints(pages)
    k, k64 = bf16(rng, (1, hkv, 128))
    c.store(k, -k, ints([(n_pages - 2) * 16 + 9]))
    kv, scale, _ = ref.store_q4(kv, scale, k64, -k64, [2 * 16 + 9])
    q, q64 = bf16(rng, (1, 8, 128))
    table = np.array([[0, 1, 2, -1]])
    want = ref.decode_q4(q64, kv, scale, table, [42], SCALE)
    check_attention(c.decode(q, ints([42])).double().cpu().numpy(), want[0], want[1], want[2], F16_HALF_STEP, want[3])
    rows = c.read(42, ints([42]))
    want = ref.read(ref.values_q4(kv, scale), table, [42], 42)
    assert (rows.k.double().cpu().numpy() == want[0]).all() and (rows.v.double().cpu().numpy() == want[1]).all()


def test_pages_past_2_to_the_26():
    """A pool of 67 million pages of one head (155 GB): written, attended and read back at its end."""
    from paged_helpers import F16_HALF_STEP, bf16, check_attention, ints
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    n_pages = 2 ** 26 + 40
    if torch.cuda.mem_get_info()[0] < 170e9:
        pytest.skip("less than 170 GB free")
    rng = np.random.default_rng(19)
    c = PagedKV(n_pages=n_pages, batch=1, nb_max=6, n_q_heads=2, n_kv_heads=1, bits=4)
    pages = [n_pages - 1, 2 ** 26, 2 ** 25 + 3, n_pages - 2, 5, 2 ** 26 - 1]
    c.table.copy_(ints([pages]))
    k, k64 = bf16(rng, (90, 1, 128))
    v, v64 = bf16(rng, (90, 1, 128))
    c.store(k, v, ints([pages[t // 16] * 16 + t % 16 for t in range(90)]))
    kv, scale, _ = ref.store_q4(np.zeros((6, 1, 2, 16, 64), np.uint8), np.zeros((6, 1, 2, 128), np.uint8), k64, v64, range(90))
    q, q64 = bf16(rng, (1, 2, 128))
    want = ref.decode_q4(q64, kv, scale, np.arange(6)[None], [90], SCALE)
    check_attention(c.decode(q, ints([90])).double().cpu().numpy(), want[0], want[1], want[2], F16_HALF_STEP, want[3])
    rows = c.read(90, ints([90]))
    assert (rows.k.double().cpu().numpy() == ref.read(ref.values_q4(kv, scale), np.arange(6)[None], [90], 90)[0]).all()
    c.check()
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("wide", [False, True])
def test_two_captured_graphs_replayed_with_other_lengths(wide):
    from paged_helpers import F16_HALF_STEP, check_attention, ints
    from q4_helpers import cache_q4

    rng = np.random.default_rng(18)
    cases, graphs = [], []
    for n in ([3000, 3000, 3000], [64, 5000, 70]):
        kv, scale, table, q, q64 = _inputs(rng, n, 2, 8, wide=wide)
        scale[scale == ref.S_NAN] = 100
        cases.append((cache_q4(kv, scale, table, 8), q, ints(n), kv, scale, table, q64))
    for c, q, ctx, *_ in cases:
        c.decode(q, ctx)
    torch.cuda.synchronize()
    for c, q, ctx, *_ in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = c.decode(q, ctx)
        graphs.append((g, out, torch.cuda.Stream()))
    for n in ([3000, 1, 0], [0, 0, 0], [17, 2999, 1], [1, 1, 1]):
        lens = [n, [n[0] // 50, n[1], n[2]]]
        for (_, _, ctx, *_), m in zip(cases, lens):
            ctx.copy_(ints(m))
        torch.cuda.synchronize()
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, kv, scale, table, q64), (_, out, _), m in zip(cases, graphs, lens):
            want = ref.decode_q4(q64, kv, scale, table, m, SCALE)
            check_attention(out.double().cpu().numpy(), want[0], want[1], want[2], F16_HALF_STEP, want[3])
