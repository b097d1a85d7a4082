"""The paged cache's 64-bit definitions against enumeration and hand examples (CPU)."""
import numpy as np
import pytest

from oracle import paged_ref as ref


def test_e4m3_rounding_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-14, 8, 4000), ref.E4M3[:0x7f],
                        (ref.E4M3[:0x7e] + ref.E4M3[1:0x7f]) / 2])  # every value and every midpoint
    x = np.concatenate([x, -x])
    x = x[np.abs(x) <= 448].astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (ref.e4m3_bytes(x.astype(np.float64)) == got).all()


def test_exponent_is_the_least():
    for amax, e in ((448.0, 0), (448.01, 1), (224.0, -1), (1.75, -8), (1.76, -7), (0.0, -60), (3.0e38, 119)):
        assert ref.exponent(amax) == e


def test_tables_by_hand():
    table = np.full((3, 4), -1)
    table[1, 0] = 9
    lens, left, start, slots, t, bits = ref.extend_tables([0, 5, 0], [17, 18, 1], np.arange(10), 8, table, 32, 10)
    # request 0 takes pages 7, 6; request 1 continues page 9 and takes 5; request 2 takes 4
    assert t.tolist() == [[7, 6, -1, -1], [9, 5, -1, -1], [4, -1, -1, -1]] and left == 4 and bits == 0
    assert start.tolist() == [0, 17, 30, 31] and lens.tolist() == [17, 18, 1]
    assert slots.tolist() == list(range(112, 128)) + [96] + list(range(149, 160)) + [80, 81] + [64, -1]
    free, n, bits = ref.release_tables([17, 18, 1], [0, 16, 1], t, np.arange(10), 4, 10)
    assert free[:7].tolist() == [0, 1, 2, 3, 7, 6, 5] and n == 7 and bits == 0


def test_store_keeps_values_when_the_scale_grows():
    kv, scale = np.zeros((1, 1, 2, 16, 128), np.uint8), np.ones((1, 1, 2))
    small, large = np.full((1, 1, 128), 1.5), np.full((1, 1, 128), 400.0)
    kv, scale, _ = ref.store(kv, scale, small, small, [0])
    assert scale[0, 0, 0] == 2.0 ** -8
    kv, scale, _ = ref.store(kv, scale, large, large, [1])
    assert scale[0, 0, 0] == 1.0 and ref.E4M3[kv[0, 0, 0, 0, 0]] == 1.5 and ref.E4M3[kv[0, 0, 0, 1, 0]] == 384.0  # a tie: even


def test_decode_equals_textbook_softmax():
    rng = np.random.default_rng(1)
    kv = ref.e4m3_bytes(rng.standard_normal((4, 1, 2, 16, 128)) * 60)
    scale, table = np.full((4, 1, 2), 2.0 ** -6), np.array([[2, 0, 3]])
    q = rng.standard_normal((1, 2, 128))
    out, _, _, _ = ref.decode(q, kv, scale, table, [37], 0.1)
    k = np.concatenate([ref.E4M3[kv[p, 0, 0]] for p in (2, 0, 3)])[:37] / 64
    v = np.concatenate([ref.E4M3[kv[p, 0, 1]] for p in (2, 0, 3)])[:37] / 64
    w = np.exp(q[0] @ k.T * 0.1)
    assert np.allclose(out[0], (w / w.sum(-1, keepdims=True)) @ v, rtol=1e-12, atol=1e-12)
    sel = np.array([[[1, 2, -1]]])
    out, _, _, _ = ref.decode(q, kv, scale, table, [37], 0.1, sel, np.array([[2]]))
    w = np.exp(q[0] @ k[16:].T * 0.1)
    assert np.allclose(out[0], (w / w.sum(-1, keepdims=True)) @ v[16:], rtol=1e-12, atol=1e-12)


def test_prompt_rows_see_the_past_of_their_own_sequence():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((7, 2, 128)), rng.standard_normal((7, 1, 128)), rng.standard_normal((7, 1, 128))
    out, _, _ = ref.prompt(q, k, v, [0, 3, 3, 6], 0.1)
    assert (out[3] == v[3, 0]).all() and (out[6] == 0).all()  # a first token; a row of no sequence
    w = np.exp(q[5] @ k[3:6, 0].T * 0.1)
    assert np.allclose(out[5], (w / w.sum(-1, keepdims=True)) @ v[3:6, 0])
