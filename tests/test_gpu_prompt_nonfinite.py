"""Packed prompts with infinities and NaN in some rows: a row's output knows only of rows up to itself."""
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


def _check(q, k, v, start, rows=None):
    """Against the definition: not-finite outputs in the same places and of the same kind, the others in tolerance."""
    from paged_helpers import BF16_HALF_STEP, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = prompt_attn(q.cuda(), k.cuda(), v.cuda(), ints(start), err=err).double().cpu().numpy()
    assert int(err) == 0
    q64, k64, v64 = (t.double().numpy() for t in (q, k, v))
    with np.errstate(invalid="ignore"):
        want = ref.prompt(q64, k64, v64, start, SCALE)[0]
    # the allowance of the finite outputs: what the roundings do does not depend on the rows that were spoilt
    _, mass, size = ref.prompt(*(np.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0) for t in (q64, k64, v64)), start, SCALE)
    fin = np.isfinite(want)
    assert (np.isfinite(got) == fin).all(), f"{int((np.isfinite(got) != fin).sum())} elements"
    assert (np.isnan(got) == np.isnan(want)).all()
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all()
    size = np.broadcast_to(size, want.shape)
    check_attention(got[fin], want[fin], mass[fin], size[fin], BF16_HALF_STEP)
    return got


def _inputs(seed, n, hkv, G):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, h, 128), generator=g).to(torch.bfloat16) for h in (hkv * G, hkv, hkv))


PLACES = [[0], [1], [77], [126, 128], [127], [255], [299], [302], [40, 41, 200, 430], list(range(60, 300, 7))]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("places", PLACES, ids=str)
@pytest.mark.parametrize("G", [1, 3, 4, 8])
def test_a_value_reaches_no_earlier_row(G, places, value):
    q, k, v = _inputs(G, 440, 2, G)
    for i, p in enumerate(places):
        v[p, i % 2, (p * 37) % 128] = value if i % 3 < 2 else -value
    _check(q, k, v, [0, 300, 305, 435])


@pytest.mark.parametrize("count", [320, 400])
def test_among_many_sequences(count):
    """Both schedules (up to 320 sequences sorted, more in their order), empty sequences among them, several
    items to a block: what was taken out goes back to the right rows."""
    rng = np.random.default_rng(count)
    lens = rng.integers(0, 12, count)
    lens[[3, count // 2]] = 150
    start = np.concatenate([[0], np.cumsum(lens)])
    n = int(start[-1])
    q, k, v = _inputs(count, n + 3, 4, 4)
    for p in rng.integers(0, n, 60):
        v[p, int(rng.integers(0, 4)), int(rng.integers(0, 128))] = [np.inf, -np.inf, np.nan][int(rng.integers(0, 3))]
    v[n:] = float("nan")
    _check(q, k, v, start.tolist())


@pytest.mark.parametrize("size", [1e19, 3e38])
def test_large_finite_values_stay(size):
    """Products of such values pass the largest bf16 where the kernel looks for infinities; the values are finite."""
    q, k, v = _inputs(40, 300, 1, 4)
    q[:] = 0  # equal weights: their sums stay finite
    v[:] = torch.where(v > 0, size, -size).to(torch.bfloat16)
    _check(q, k, v, [0, 200, 299])


def test_small_values_stay():
    """Values of 2^-100, whose products with the weights lie below fp32's normal range."""
    from paged_helpers import BF16_HALF_STEP, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    q, k, v = _inputs(41, 300, 1, 4)
    small = (v.float() * 2.0 ** -100).to(torch.bfloat16)
    got = prompt_attn(q.cuda(), k.cuda(), small.cuda(), ints([0, 300])).double().cpu().numpy() * 2.0 ** 100
    want, mass, size = ref.prompt(*(t.double().numpy() for t in (q, k, v)), [0, 300], SCALE)
    # half of fp32's smallest step, 2^-150, is 2^-16 of a weight of 2^-34 times 2^-100: inside what the sums are allowed
    check_attention(got, want, mass, size, BF16_HALF_STEP)


@pytest.mark.parametrize("G", [1, 4])
def test_rows_of_values_that_are_all_nan(G):
    q, k, v = _inputs(9, 700, 1, G)
    v[333:] = float("nan")
    _check(q, k, v, [0, 600, 690])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("G", [1, 4])
def test_a_key_reaches_no_earlier_row(G, value):
    q, k, v = _inputs(G + 20, 300, 1, G)
    k[[5, 130, 290], 0, 3] = value
    _check(q, k, v, [0, 260, 299])


def test_a_query_spoils_its_row_alone():
    q, k, v = _inputs(30, 300, 1, 4)
    q[[0, 64, 280], [0, 3, 1], 7] = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=torch.bfloat16)
    _check(q, k, v, [0, 150, 299])


def test_scores_of_minus_infinity_have_no_weight():
    """The first 200 keys' scores pass the lowest fp32 and are -inf: rows that see nothing else are NaN
    (0 / 0), later rows attend the other keys, whose scores are low too."""
    from paged_helpers import BF16_HALF_STEP, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    n = 330
    q, k, v = _inputs(31, n, 1, 2)
    q[:] = 0
    q[:, :, 0] = 2.0 ** 100
    k[:] = 0
    k[:, 0, 0] = -(2.0 ** -90)  # a score of -1024 * scale
    k[:200, 0, 0] = -(2.0 ** 100)
    got = prompt_attn(q.cuda(), k.cuda(), v.cuda(), ints([0, n])).double().cpu().numpy()
    q64, k64, v64 = (t.double().numpy() for t in (q, k, v))
    # -inf weighs nothing: the definition over the keys from 200 on
    want, mass, size = ref.prompt(q64[200:], k64[200:], v64[200:], [0, n - 200], SCALE)
    check_attention(got[200:], want, mass, size, BF16_HALF_STEP)
    assert np.isnan(got[:200]).all()
