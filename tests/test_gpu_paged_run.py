"""The paged cache's operators as a serving loop uses them, together with the sparse path's selection."""
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


def test_prompts_then_decode_steps():
    """Two layers: packed prompts (attended, stored), then decode steps, then a request leaves and
    another takes its pages; every output and the cache's state against the definitions."""
    from paged_helpers import BF16_HALF_STEP, F16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import PagedKV, prompt_attn

    rng = np.random.default_rng(0)
    hkv, G, layers, n_pages = 2, 4, 2, 40
    c = PagedKV(n_pages=n_pages, batch=3, nb_max=16, n_q_heads=hkv * G, n_kv_heads=hkv, layers=layers)
    c.kv.zero_()
    lens = np.array([70, 1, 33])
    table, free, n_free = c.table.cpu().numpy(), c.free.cpu().numpy(), n_pages
    pages = [[np.zeros((n_pages, hkv, 2, 16, 128), np.uint8), np.ones((n_pages, hkv, 2))] for _ in range(layers)]

    def store(layer, plan, slots, rows):
        k, k64 = bf16(rng, (rows, hkv, 128))
        v, v64 = bf16(rng, (rows, hkv, 128), 2.0)
        c.store(k, v, plan.slot_map, layer)
        pages[layer] = list(ref.store(*pages[layer], k64, v64, slots)[:2])
        assert (c.kv[layer].cpu().numpy() == pages[layer][0]).all()
        return k, v, k64, v64

    rows = int(lens.sum()) + 6
    plan = c.extend(ints(lens), rows)
    _, n_free, start, slots, table, _ = ref.extend_tables(np.zeros(3, int), lens, free, n_free, table, rows, n_pages)
    for layer in range(layers):
        k, v, k64, v64 = store(layer, plan, slots, rows)
        q, q64 = bf16(rng, (rows, hkv * G, 128))
        out = prompt_attn(q, k, v, plan.row_start).double().cpu().numpy()
        want, mass, size = ref.prompt(q64, k64, v64, start, SCALE)
        check_attention(out, want, mass, size, BF16_HALF_STEP)
    c.commit(plan)

    for step in range(20):
        if step == 10:  # request 0 leaves; its place is taken by one of 50 tokens
            c.release(ints([0, lens[1], lens[2]]))
            free, n_free, _ = ref.release_tables(lens, [0, lens[1], lens[2]], table, free, n_free, n_pages)
            lens[0] = 0
        new = lens + 1 if step != 10 else np.array([50, lens[1] + 1, lens[2] + 1])
        rows = int((new - lens).sum())
        plan = c.extend(ints(new), rows)
        lens, n_free, _, slots, table, _ = ref.extend_tables(lens, new, free, n_free, table, rows, n_pages)
        for layer in range(layers):
            store(layer, plan, slots, rows)
            q, q64 = bf16(rng, (3, hkv * G, 128))
            out = c.decode(q, plan.lens, layer).double().cpu().numpy()
            want = ref.decode(q64, *pages[layer], table, lens, SCALE)
            check_attention(out, want[0], want[1], want[2], F16_HALF_STEP, want[3])
        c.commit(plan)
    c.check()


def test_the_sparse_path_selects_for_the_paged_cache():
    """oasis_score_blocks and oasis_topk_select choose blocks from the bf16 keys; the 8-bit pages of
    those blocks are attended.  The budget covers the whole context of one request and not the other's."""
    from paged_helpers import F16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300 import binding as B
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    rng = np.random.default_rng(1)
    hkv, G, nb_max, kb, n_la = 8, 4, 64, 24, 2
    ctx = np.array([1000, 300])
    k, k64 = bf16(rng, (2, nb_max * 16, hkv, 128))
    v, v64 = bf16(rng, (2, nb_max * 16, hkv, 128))
    q, q64 = bf16(rng, (2, hkv * G, 128))
    q_la = (q[:, None] + 0.3 * torch.randn(2, n_la, hkv * G, 128, device="cuda")).to(torch.bfloat16)
    shape = B.Shape.of(B=2, Hq=hkv * G, Hkv=hkv, nb_max=nb_max, n_la=n_la, Kb=kb, P=kb)
    scores = torch.zeros((2, hkv, nb_max, 2), device="cuda")
    sel = torch.zeros((2, hkv, kb), dtype=torch.int32, device="cuda")
    nsel = torch.zeros((2, hkv), dtype=torch.int32, device="cuda")
    keys = k.transpose(1, 2).contiguous()
    c = PagedKV(n_pages=2 * nb_max, batch=2, nb_max=nb_max, n_q_heads=hkv * G, n_kv_heads=hkv)
    plan = c.extend(ints(ctx), int(ctx.sum()))
    rows = [k[b, :n] for b, n in enumerate(ctx)], [v[b, :n] for b, n in enumerate(ctx)]
    c.store(torch.cat(rows[0]), torch.cat(rows[1]), plan.slot_map)
    c.commit(plan)
    B.oasis_score_blocks(shape, keys, c.lens, q_la, scores)
    B.oasis_topk_select(shape, scores, keys, q_la, c.lens, sel, nsel)
    out = c.decode(q, sel=sel, nsel=nsel).double().cpu().numpy()
    c.check()
    assert nsel[0].eq(kb).all() and nsel[1].eq(19).all()
    want = ref.decode(q64, c.kv[0].cpu().numpy(), c.scale[0].double().cpu().numpy(), c.table.cpu().numpy(), ctx, SCALE,
                      sel.cpu().numpy(), nsel.cpu().numpy())
    check_attention(out, want[0], want[1], want[2], F16_HALF_STEP, want[3])
    dense = c.decode(q).double().cpu().numpy()
    assert np.abs(dense[1] - out[1]).max() <= 2.0 ** -7 * np.abs(out[1]).max()  # all its blocks, in another order or split


def test_calls_that_follow_closely_see_what_the_call_before_wrote():
    """A kernel is launched while its predecessor still drains: a run without a pause gives the bits of
    a run that waits for the device after every call (outputs, pages and scales).  Values of very
    different sizes make the stores rescale pages that the step before attended."""
    from sparse_decode_attention_oasis_gb300.paged import PagedKV, prompt_attn

    batch, hkv, hq, steps = 24, 8, 32, 40
    g = torch.Generator(device="cuda").manual_seed(3)

    def rows(n, heads, size=1.0):
        return (torch.randn((n, heads, 128), device="cuda", generator=g) * size).bfloat16()

    def run(cache, pause):
        outs = []
        plan = cache.extend(lens, n)
        pause()
        outs.append(prompt_attn(q, k, v, plan.row_start))
        pause()
        cache.store(k, v, plan.slot_map)
        pause()
        cache.commit(plan)
        for kk, vv, qq in new:
            longer = cache.lens + 1
            pause()
            plan = cache.extend(longer, batch)
            pause()
            cache.store(kk, vv, plan.slot_map)
            pause()
            outs.append(cache.decode(qq, plan.lens))
            pause()
            cache.commit(plan)
        cache.check()
        return outs

    for _ in range(4):
        lens = torch.randint(1, 300, (batch,), dtype=torch.int32, device="cuda", generator=g)
        n = int(lens.sum())
        q, k, v = rows(n, hq), rows(n, hkv), rows(n, hkv)
        new = [(rows(batch, hkv, 2.0 ** (i % 9 - 4)), rows(batch, hkv, 2.0 ** (i * 5 % 11 - 5)), rows(batch, hq))
               for i in range(steps)]
        caches = [PagedKV(n_pages=batch * 22, batch=batch, nb_max=22, n_q_heads=hq, n_kv_heads=hkv) for _ in range(2)]
        for c in caches:
            c.kv.zero_()
        torch.cuda.synchronize()
        got = run(caches[0], lambda: None)
        want = run(caches[1], torch.cuda.synchronize)
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"call {i}"
        assert torch.equal(caches[0].kv, caches[1].kv) and torch.equal(caches[0].scale, caches[1].scale)
