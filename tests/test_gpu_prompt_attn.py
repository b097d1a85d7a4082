"""Causal attention over packed prompts against the 64-bit definition."""
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


def _start(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)])


def _check(lens, hkv, G, seed=0, pad=0, first=0, q_size=1.0, scale=None, rows=None):
    """`rows`: rows of long sequences that are compared (the definition costs n^2)."""
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(seed)
    n, hq = first + sum(lens) + pad, hkv * G
    buf, buf64 = bf16(rng, (n, hq + 2 * hkv, 128))
    buf[:, :hq] *= q_size
    buf64 = buf.double().cpu().numpy()
    dev = buf.clone()
    dev[:first] = float("nan")  # rows of no sequence
    dev[first + sum(lens):] = float("nan")
    out = torch.full((n, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    start = _start(lens, first)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = prompt_attn(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], ints(start), scale=scale, out=out, err=err)
    assert got is out and int(err) == 0
    got = out.double().cpu().numpy()
    assert (got[:first] == 7).all() and (got[first + sum(lens):] == 7).all()
    q, k, v = buf64[:, :hq], buf64[:, hq:hq + hkv], buf64[:, hq + hkv:]
    if rows is None:
        want, mass, size = ref.prompt(q, k, v, start, scale or SCALE)
        keep = np.arange(first, first + sum(lens))
        check_attention(got[keep], want[keep], mass[keep], size[keep], BF16_HALF_STEP)
    else:
        for a, i in rows:  # row i of the sequence that starts at row a
            for h in range(hkv):
                r = slice(h * G, h * G + G)
                want, mass, size, _ = ref._softmax_rows(q[a + i, r], k[a:a + i + 1, h], v[a:a + i + 1, h], scale or SCALE)
                check_attention(got[a + i, r], want, mass, np.float64(size), BF16_HALF_STEP)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_group_sizes(G):
    _check([1, 40, 130, 17, 300], 2, G, seed=G)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31, 33], [63, 64, 65], [127, 128, 129], [255, 256, 257],
                                  [0, 5, 0, 0, 3, 0], [0], [1] * 70, [383, 1, 385], [511, 513]])
@pytest.mark.parametrize("G", [1, 4])
def test_lengths(lens, G):
    _check(lens, 1, G, seed=sum(lens) + G, pad=3)


@pytest.mark.parametrize("G,hkv", [(4, 2), (8, 1), (1, 3), (7, 1)])
def test_long(G, hkv):
    n = 3001
    rows = [(0, i) for i in (0, 1, 127, 128, 129, 1000, 2047, 2048, n - 2, n - 1)] + [(n, i) for i in (0, 500, 1029)]
    _check([n, 1030], hkv, G, seed=n + G, pad=1, rows=rows)


@pytest.mark.parametrize("count", [320, 321, 700])
def test_many_sequences(count):
    """Both schedules: up to 320 sequences sorted, more in their order; empty ones among them."""
    rng = np.random.default_rng(count)
    lens = [int(n) for n in rng.integers(0, 9, count)]
    lens[count // 2] = 600
    _check(lens, 1, 4, seed=count, pad=2)


def test_rows_before_and_behind_are_left():
    _check([37, 5], 2, 4, seed=1, pad=200, first=11)


@pytest.mark.parametrize("q_size", [0.0, 1e-3, 20.0, 300.0])
def test_query_sizes(q_size):
    """From equal weights to a softmax that takes one token."""
    _check([200, 9], 1, 4, seed=2, q_size=q_size)


def test_given_scale():
    _check([90], 1, 2, seed=3, scale=0.7)


def test_scores_that_grow_and_fall():
    """Keys whose scores climb by far more than the slack of a running maximum, then fall."""
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(4)
    n = 900
    q, _ = bf16(rng, (n, 2, 128))
    q[:] = 1.0
    size = torch.cat([torch.linspace(-8, 8, n // 2), torch.linspace(8, -8, n - n // 2)])
    k = (size[:, None, None] * torch.ones(n, 1, 128)).to(torch.bfloat16)
    v, v64 = bf16(rng, (n, 1, 128))
    got = prompt_attn(q, k.cuda(), v, ints([0, n])).double().cpu().numpy()
    want, mass, sz = ref.prompt(q.double().cpu().numpy(), k.double().numpy(), v64, [0, n], SCALE)
    check_attention(got, want, mass, sz, BF16_HALF_STEP)


def test_sequences_that_break_the_rule_are_skipped():
    from paged_helpers import BF16_HALF_STEP, bf16, check_attention, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(5)
    q, q64 = bf16(rng, (60, 4, 128))
    k, k64 = bf16(rng, (60, 2, 128))
    v, v64 = bf16(rng, (60, 2, 128))
    out = torch.full((60, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # [-4, 10) and [30, 20) break it, [20, 61) ends behind the rows; [10, 30) stands
    prompt_attn(q, k, v, ints([-4, 10, 30, 20, 61]), out=out, err=err)
    assert int(err) == 8
    got = out.double().cpu().numpy()
    want, mass, size = ref.prompt(q64, k64, v64, [10, 30], SCALE)
    check_attention(got[10:30], want[10:30], mass[10:30], size[10:30], BF16_HALF_STEP)
    assert (got[:10] == 3).all() and (got[30:] == 3).all()


def test_no_rows_and_a_given_default_output():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(6)
    q, _ = bf16(rng, (12, 4, 128))
    k, _ = bf16(rng, (12, 4, 128))
    assert prompt_attn(q[:0], k[:0], k[:0], ints([0, 0])).shape == (0, 4, 128)
    out = prompt_attn(q, k, k, ints([0, 5]))
    assert (out[5:] == 0).all()
    assert torch.equal(out[0], k[0])  # a first token attends itself alone


def test_refusals():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.binding import OasisError
    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(7)
    q, _ = bf16(rng, (12, 4, 128))
    k, _ = bf16(rng, (12, 2, 128))
    s = ints([0, 12])
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:5]), dict(v=k[:, :1]), dict(row_start=s.long()), dict(row_start=s[:1]),
                dict(out=q.float()), dict(q=q.transpose(0, 1)), dict(err=s), dict(k=k.cpu())):
        with pytest.raises(ValueError):
            prompt_attn(**{"q": q, "k": k, "v": k, "row_start": s, **bad})
    for bad in (dict(q=q[:, :3]), dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(OasisError):
            prompt_attn(**{"q": q, "k": k, "v": k, "row_start": s, **bad})


def test_two_streams_at_once():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(9)
    cases = []
    for n, cut in ((3000, 1100), (2500, 7)):
        q, _ = bf16(rng, (n, 8, 128))
        k, _ = bf16(rng, (n, 2, 128))
        cases.append((q, k, ints([0, cut, n]), torch.cuda.Stream()))
    alone = [prompt_attn(q, k, k, s) for q, k, s, _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for q, k, s, st in cases:
            with torch.cuda.stream(st):
                outs.append(prompt_attn(q, k, k, s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, alone))


def test_captured_and_replayed_with_other_lengths():
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    rng = np.random.default_rng(8)
    q, _ = bf16(rng, (400, 4, 128))
    k, _ = bf16(rng, (400, 2, 128))
    start = ints([0, 10, 400])
    out = torch.zeros((400, 4, 128), dtype=torch.bfloat16, device="cuda")
    prompt_attn(q, k, k, start, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prompt_attn(q, k, k, start, out=out)
    for s in ([0, 10, 400], [0, 300, 350], [0, 0, 400]):
        start.copy_(ints(s))
        want = prompt_attn(q, k, k, start, out=torch.zeros_like(out))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
