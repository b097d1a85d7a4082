"""The 4-bit store on the GPU against the 64-bit definition: codes and scale bytes equal.

The definition has one right answer for every byte, so nothing is tolerated."""
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


def _bf16(rng, shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).to(torch.bfloat16)


def _run(k, v, slots, n_pages, seed=0):
    """k, v: bf16 on the CPU [rows][hkv][128]; the pool holds other bytes before, which have to stay."""
    from paged_helpers import ints
    from q4_helpers import cache_q4, random_pages_q4

    hkv = k.shape[1]
    kv, scale = random_pages_q4(np.random.default_rng(seed), n_pages, hkv)
    c = cache_q4(kv, scale, np.zeros((1, 1), int), hkv)
    c.store(k.cuda(), v.cuda(), ints(slots))
    want_kv, want_scale, bits = ref.store_q4(kv, scale, k.double().numpy(), v.double().numpy(), slots)
    assert (c.scale[0].cpu().numpy() == want_scale).all()
    assert (c.kv[0].cpu().numpy() == want_kv).all()
    assert int(c.err) == bits
    return c


@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("rows", [1, 2, 7, 31, 32, 500])
def test_rows_in_any_order(hkv, rows):
    rng = np.random.default_rng(rows * 10 + hkv)
    n_pages = rows // 8 + 2
    slots = rng.permutation(n_pages * 16)[:rows]
    slots[rng.random(rows) < 0.1] = -1
    _run(_bf16(rng, (rows, hkv, 128)), _bf16(rng, (rows, hkv, 128), 3.0), slots, n_pages)


def test_a_long_call():
    """More rows than warps at a time: several rows to a warp, the last group of them not full."""
    rng = np.random.default_rng(1)
    rows, hkv = 3001, 8
    _run(_bf16(rng, (rows, hkv, 128)), _bf16(rng, (rows, hkv, 128)), np.arange(rows) + 5, 190)


def test_every_bf16_value_that_is_a_number():
    """Each beside zeros alone, and each as the smaller one of a group of its own size's neighbours."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[~torch.isnan(x.float())]
    n = -(-x.numel() // 8)
    k = torch.zeros(n, 8, 16, dtype=torch.bfloat16)
    k.view(-1, 16)[torch.arange(x.numel()), torch.arange(x.numel()) % 16] = x
    g = torch.Generator().manual_seed(2)
    size = 2.0 ** torch.randint(0, 9, (n, 8, 1), generator=g)
    v = torch.zeros(n, 8, 16)
    v.view(-1, 16)[torch.arange(x.numel())] = x.float()[:, None]
    v = (v * torch.randn((n, 8, 16), generator=g) / size).to(torch.bfloat16)
    v[torch.isnan(v.float())] = 0
    v.view(-1, 16)[torch.arange(x.numel()), 3] = x
    _run(k.view(n, 1, 128), v.view(n, 1, 128), np.arange(n), -(-n // 16))


def test_ties():
    """Every tie of the codes, for every scale: values at 1/4 steps of it beside its 6."""
    s = ref.scale_value(np.arange(1, ref.S_HIGH + 1))
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0])
    x = torch.from_numpy(s[:, None] * mids)
    k = torch.zeros(len(s), 1, 128, dtype=torch.bfloat16)
    k[:, 0, 16:32] = x.to(torch.bfloat16)
    assert (k[:, 0, 16:32].double() == x).all()
    c = _run(k, -k, np.arange(len(s)), 15)
    assert c.kv[0].any()


def test_zeros_infinities_and_nan():
    rng = np.random.default_rng(3)
    k, v = _bf16(rng, (6, 2, 128)), _bf16(rng, (6, 2, 128))
    k[0, 0, :32], k[1, 1, 5], k[2, 0, 7], v[3, 1, 64] = 0, float("inf"), float("-inf"), float("nan")
    v[4], k[5, 0, 90], k[5, 0, 91] = -0.0, float("nan"), float("inf")
    c = _run(k, v, np.arange(6), 1)
    got = ref.values_q4(c.kv[0].cpu().numpy(), c.scale[0].cpu().numpy())
    assert got[0, 1, 0, 1, 5] == 61440 and got[0, 0, 0, 2, 7] == -61440
    assert np.isnan(got[0, 1, 1, 3, 64:80]).all() and np.isnan(got[0, 0, 0, 5, 80:96]).all()
    assert np.isfinite(got).sum() == got.size - 32


def test_slots_outside_the_pool_are_skipped_and_flagged():
    rng = np.random.default_rng(4)
    k, v = _bf16(rng, (5, 2, 128)), _bf16(rng, (5, 2, 128))
    _run(k, v, np.array([3, 48, -2, 2 ** 31 - 1, 40]), 3)
    _run(k, v, np.array([-1] * 5), 3)


def test_slices_of_a_fused_buffer():
    from paged_helpers import ints
    from q4_helpers import cache_q4, random_pages_q4

    rng = np.random.default_rng(5)
    wide = _bf16(rng, (40, 9, 128))
    kv, scale = random_pages_q4(rng, 4, 2)
    c = cache_q4(kv, scale, np.zeros((1, 1), int), 2)
    dev = wide.cuda()
    c.store(dev[:, 3:5], dev[:, 7:9], ints(np.arange(40) + 10))
    want = ref.store_q4(kv, scale, wide[:, 3:5].double().numpy(), wide[:, 7:9].double().numpy(), np.arange(40) + 10)
    assert (c.kv[0].cpu().numpy() == want[0]).all() and (c.scale[0].cpu().numpy() == want[1]).all()


@pytest.mark.parametrize("first,stride", [(8, 1024 * 2), (0, 1024 * 2 + 8), (24, 1024 * 2 + 40)])
@pytest.mark.parametrize("rows", [5, 4003])
def test_rows_on_16_byte_boundaries_only(rows, first, stride):
    from paged_helpers import ints
    from q4_helpers import cache_q4, random_pages_q4

    rng = np.random.default_rng(rows)
    n_pages = rows // 16 + 1
    buf = _bf16(rng, (rows * stride + 1024,))
    k = buf.as_strided((rows, 8, 128), (stride, 128, 1), first)
    v = buf.as_strided((rows, 8, 128), (stride, 128, 1), first + 512)
    kv, scale = random_pages_q4(rng, n_pages, 8)
    c = cache_q4(kv, scale, np.zeros((1, 1), int), 8)
    slots = rng.permutation(n_pages * 16)[:rows]
    on_gpu = buf.cuda()
    c.store(on_gpu.as_strided(k.shape, k.stride(), first), on_gpu.as_strided(k.shape, k.stride(), first + 512), ints(slots))
    want_kv, want_scale, _ = ref.store_q4(kv, scale, k.double().numpy(), v.double().numpy(), slots)
    assert (c.scale[0].cpu().numpy() == want_scale).all() and (c.kv[0].cpu().numpy() == want_kv).all()
    assert int(c.err) == 0


def test_refusals():
    from paged_helpers import ints
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    c = PagedKV(n_pages=2, batch=1, nb_max=2, n_q_heads=2, n_kv_heads=2, layers=2, bits=4)
    k, slots = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda"), ints([0, 1, 2])
    for bad in (dict(k=k.float()), dict(k=k[:2]), dict(v=k[:, :1]), dict(slot_map=slots.long()), dict(layer=2), dict(layer=-1)):
        with pytest.raises(ValueError):
            c.store(**{"k": k, "v": k, "slot_map": slots, **bad})
    with pytest.raises(ValueError):
        PagedKV(n_pages=2, batch=1, nb_max=2, n_q_heads=2, n_kv_heads=2, bits=2)
    with pytest.raises(ValueError):
        c.adopt(scale=torch.ones((2, 2, 2, 2), device="cuda"))
    c.store(k[:0], k[:0], slots[:0])
