"""The 8-bit store on the GPU against the 64-bit definition: bytes and scales equal.

The scale is a power of two, so x * 2^-e is exact and the one rounding, to the nearest e4m3,
has one right answer."""
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


def _pool(rng, n_pages, hkv):
    kv = ref.e4m3_bytes(rng.standard_normal((n_pages, hkv, 2, 16, 128)) * 50)
    return kv, 2.0 ** rng.integers(-8, 3, (n_pages, hkv, 2)).astype(np.float64)


def _run(kv, scale, k, v, slots, hkv):
    """k, v: bf16 CPU tensors [rows][hkv][128]."""
    from paged_helpers import cache_of, ints

    c = cache_of(kv, scale, np.zeros((1, 1), int), hkv)
    c.store(k.cuda(), v.cuda(), ints(slots))
    want_kv, want_scale, bits = ref.store(kv, scale, k.double().numpy(), v.double().numpy(), np.asarray(slots))
    got_scale = c.scale[0].cpu().numpy().astype(np.float64)
    assert (got_scale == want_scale).all()
    assert (c.kv[0].cpu().numpy() == want_kv).all()
    assert int(c.err) == bits
    return c


def _bf16(rng, shape, size=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).to(torch.bfloat16)


def _slots(rng, runs, n_pages, gaps=True):
    """Slots of runs (first position, rows) on distinct pages, some rows skipped between them."""
    slots, pages = [], rng.permutation(n_pages)
    for p, (pos, n) in zip(pages, runs):
        slots += list(range(p * 16 + pos, p * 16 + pos + n))
        if gaps and rng.random() < 0.3:
            slots += [-1] * int(rng.integers(1, 4))
    return slots


@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("runs", [[(0, 1)], [(0, 16)], [(15, 1)], [(5, 11)], [(0, 16), (0, 16), (0, 3), (7, 2), (1, 15)],
                                  [(3, 1)] * 7, [(0, 1)] * 40])
def test_runs(hkv, runs):
    rng = np.random.default_rng(hkv * 100 + len(runs))
    kv, scale = _pool(rng, 50, hkv)
    slots = _slots(rng, runs, 50)
    shape = (len(slots), hkv, 128)
    _run(kv, scale, _bf16(rng, shape), _bf16(rng, shape, 4.0), slots, hkv)


@pytest.mark.parametrize("rows", [900, 4000])  # both sides of the rule for rows per warp, with its smaller runs
def test_many_rows(rows):
    rng = np.random.default_rng(rows)
    kv, scale = _pool(rng, 600, 8)
    runs, n = [], 0
    while n < rows - 16 and len(runs) < 590:
        pos = int(rng.integers(0, 16)) if rng.random() < 0.3 else 0
        runs.append((pos, int(rng.integers(1, 17 - pos)) if rows < 1000 else 16 - pos))
        n += runs[-1][1]
    slots = _slots(rng, runs, 600)
    k = _bf16(rng, (len(slots), 8, 128))
    _run(kv, scale, k, _bf16(rng, k.shape, 0.1), slots, 8)


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-17, 1.0, 1e20, 1e38])
def test_sizes(size):
    """From below the smallest scale (values that vanish) to the largest bf16."""
    rng = np.random.default_rng(3)
    kv, scale = _pool(rng, 8, 2)
    slots = _slots(rng, [(0, 16), (4, 3), (0, 1)], 8)
    k = _bf16(rng, (len(slots), 2, 128), size)
    v = k.clone()
    v[:, :, ::3] = 0
    v[0] = 0
    _run(kv, scale, k.nan_to_num(posinf=1e38, neginf=-1e38), v.nan_to_num(posinf=1e38, neginf=-1e38), slots, 2)


def test_a_growing_scale_moves_earlier_tokens():
    rng = np.random.default_rng(4)
    kv, scale = _pool(rng, 4, 1)
    scale[:] = 2.0 ** -20
    for growth in (1.0, 2.0 ** 8, 2.0 ** 12, 2.0 ** 40, 2.0 ** 130):
        k = _bf16(rng, (2, 1, 128), 2.0 ** -15) * growth
        _run(kv, scale, k, -k, [1 * 16 + 9, 1 * 16 + 10], 1)


def test_a_page_filled_token_by_token():
    rng = np.random.default_rng(5)
    from paged_helpers import cache_of, ints

    kv, scale = _pool(rng, 3, 2)
    c = cache_of(kv, scale, np.zeros((1, 1), int), 2)
    for t in range(16):
        k, v = _bf16(rng, (1, 2, 128), 1.2 ** t), _bf16(rng, (1, 2, 128), 3.0 ** (t % 5))
        c.store(k.cuda(), v.cuda(), ints([2 * 16 + t]))
        kv, scale, _ = ref.store(kv, scale, k.double().numpy(), v.double().numpy(), np.array([2 * 16 + t]))
        assert (c.kv[0].cpu().numpy() == kv).all() and (c.scale[0].cpu().numpy() == scale).all()


def test_ties_and_every_value():
    """All e4m3 values and all their midpoints: the midpoints fit bf16's 8 significant bits."""
    both = np.concatenate([ref.E4M3[:0x7f], (ref.E4M3[:0x7e] + ref.E4M3[1:0x7f]) / 2])
    x = np.concatenate([both, -both, np.zeros(6)])
    x = np.resize(x, (4, 1, 128))
    k = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    assert (k.double().numpy() == x).all()
    kv, scale = np.zeros((2, 1, 2, 16, 128), np.uint8), np.ones((2, 1, 2))
    _run(kv, scale, k, -k, [0, 1, 2, 3], 1)


def test_bad_slots_are_skipped():
    rng = np.random.default_rng(6)
    kv, scale = _pool(rng, 4, 2)
    slots = [4 * 16, 5, 6, 6, 7, 9, -1, -5, 2 ** 31 - 1, 30, 31, 32, 33, 35]
    k = _bf16(rng, (len(slots), 2, 128))
    _run(kv, scale, k, k, slots, 2)


def test_non_finite_rows_stay_in_their_page():
    rng = np.random.default_rng(7)
    kv, scale = _pool(rng, 4, 1)
    k = _bf16(rng, (3, 1, 128))
    k[0, 0, 5] = float("inf")
    k[1, 0, 6] = float("nan")
    from paged_helpers import cache_of, ints

    c = cache_of(kv, scale, np.zeros((1, 1), int), 1)
    c.store(k.cuda(), k.cuda(), ints([0, 1, 16]))
    got = c.kv[0].cpu().numpy()
    assert (got[2:] == kv[2:]).all() and (got[1, :, :, 1:] == kv[1, :, :, 1:]).all()
    assert (c.scale[0, 0].cpu().numpy() == 2.0 ** 119).all()
    assert got[0, 0, 0, 0, 5] == 0x7e and got[0, 0, 0, 1, 6] & 0x7f == 0x7f  # saturated, NaN


def test_slices_of_one_buffer():
    rng = np.random.default_rng(8)
    kv, scale = _pool(rng, 6, 2)
    slots = _slots(rng, [(0, 16), (3, 9)], 6, gaps=False)
    buf = _bf16(rng, (len(slots), 9, 128))
    from paged_helpers import cache_of, ints

    c = cache_of(kv, scale, np.zeros((1, 1), int), 2)
    dev = buf.cuda()
    c.store(dev[:, 4:6], dev[:, 7:9], ints(slots))
    want = ref.store(kv, scale, buf[:, 4:6].double().numpy(), buf[:, 7:9].double().numpy(), np.array(slots))
    assert (c.kv[0].cpu().numpy() == want[0]).all() and (c.scale[0].cpu().numpy() == want[1]).all()


def test_layers_are_apart():
    from paged_helpers import ints

    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    c = PagedKV(n_pages=3, batch=1, nb_max=2, n_q_heads=2, n_kv_heads=2, layers=3)
    c.kv.zero_()
    k = torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    c.store(k, k, ints([16, 17]), layer=1)
    assert c.kv[0].any() == 0 and c.kv[2].any() == 0 and c.kv[1, 1].any()
    for bad in (-1, 3):
        with pytest.raises(ValueError):
            c.store(k, k, ints([16, 17]), layer=bad)
    with pytest.raises(ValueError):
        c.store(k.float(), k, ints([16, 17]))
    with pytest.raises(ValueError):
        c.store(k[:, :1], k, ints([16, 17]))
    with pytest.raises(ValueError):
        c.store(k.transpose(1, 2).contiguous().transpose(1, 2), k, ints([16, 17]))
