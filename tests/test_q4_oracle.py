"""Pins of the 4-bit pages' definitions, and of the arithmetic that the store rests on (CPU)."""
from fractions import Fraction

import numpy as np

from oracle import paged_ref as ref


def test_scale_bytes_are_the_halves_of_their_shifted_bits():
    b = np.arange(256)
    halves = (b << 7).astype(np.uint16).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(ref.scale_value(b), halves)
    assert ref.scale_value(1) == 2.0 ** -17 and ref.scale_value(8) == 2.0 ** -14 and ref.scale_value(ref.S_HIGH) == 10240


def test_stored_values_are_halves_and_bf16_values():
    """code * scale for every pair: exact in fp16 (what the products take) and in bf16 (what is read back)."""
    v = ref.E2M1[:, None] * ref.scale_value(np.arange(ref.S_HIGH + 1))
    assert (v.astype(np.float16).astype(np.float64) == v).all()
    bits = v.astype(np.float32).view(np.uint32)
    assert (bits & 0xffff == 0).all() and (v.astype(np.float32) == v).all()


def test_the_scale_is_the_least_one():
    rng = np.random.default_rng(0)
    bits = np.concatenate([rng.integers(0, 0x7f80, 3000), np.arange(0x3f00, 0x4100)])
    for x in (bits << 16).astype(np.uint32).view(np.float32).astype(np.float64):
        b = int(ref.scale_byte(x))
        s = ref.scale_value(np.arange(ref.S_HIGH + 1))
        assert b == ref.S_HIGH or x <= 6 * s[b]
        assert b == 0 or x > 6 * s[b - 1]
    assert ref.scale_byte(0.0) == 0 and ref.scale_byte(1e30) == ref.S_HIGH == ref.scale_byte(np.inf)


def test_codes_are_the_nearest_ties_to_even():
    y = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.001, 100.0, -0.25, -0.2501, -2.5, 0.0, -0.0])
    assert ref.e2m1_codes(y).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 0, 9, 12, 0, 0]
    for y in np.random.default_rng(1).uniform(-7, 7, 2000):
        c = int(ref.e2m1_codes(y))
        assert abs(ref.E2M1[c] - np.clip(y, -6, 6)) == np.abs(ref.E2M1 - np.clip(y, -6, 6)).min()


def test_the_quotient_formed_by_a_reciprocal_has_the_right_code():
    """x * (1 / s) in fp32, rounded to a multiple of 2^-16: the same code as the exact quotient's, for every
    significand of x and of s and every exponent between them that matters (both are scaled by powers of two),
    with a reciprocal that is off by up to 2^-22."""
    x = np.arange(1, 256)
    for s in range(1, 16):  # subnormal scales have fewer bits
        for off in (-2.0 ** -22, 0.0, 2.0 ** -22):
            inv = np.float32(1.0 / s * (1 + off))
            for e in range(-12, 8):
                xs = x * 2.0 ** e
                keep = xs / s <= 6
                product = xs[keep].astype(np.float32).astype(np.float64) * np.float64(inv)  # exact: 8 + 24 bits
                y = (product + 192.0).astype(np.float32) - np.float32(192.0)  # one rounding, as a fused multiply-add's
                exact = np.array([float(Fraction(v) / s) for v in xs[keep].tolist()])
                np.testing.assert_array_equal(ref.e2m1_codes(y.astype(np.float64)), ref.e2m1_codes(exact))


def test_the_scale_formed_by_a_product_is_the_least_one():
    """amax * fl(1/6) in fp32 for every bf16 amax, then the next scale at or above it."""
    a = (np.arange(0x7f80) << 16).astype(np.uint32).view(np.float32)
    r = a * np.float32(1 / 6)
    low = np.ceil(r.astype(np.float64) * 2.0 ** 17)
    normal = ((r.view(np.uint32).astype(np.int64) + 0xfffff) >> 20) - 896
    got = np.where(r < 2.0 ** -14, low, np.minimum(normal, ref.S_HIGH))
    np.testing.assert_array_equal(got, ref.scale_byte(a.astype(np.float64)))


def test_values_follow_the_layout():
    """One token, one group: bytes put by hand."""
    kv, scale = np.zeros((1, 1, 2, 16, 64), np.uint8), np.zeros((1, 1, 2, 128), np.uint8)
    kv[0, 0, 0, 5, 9] = 0xa7          # key of token 5: dimension 18 is code 7, dimension 19 code 10
    scale[0, 0, 0, 5 * 8 + 1] = 128   # its group 1: 2.0
    kv[0, 0, 1, 14, 63] = 0x3c        # value of token 14: dimension 126 is code 12, 127 code 3
    scale[0, 0, 1, 7 * 16 + 14] = 120  # group 7 of token 14: 1.0
    v = ref.values_q4(kv, scale)
    assert v[0, 0, 0, 5, 18] == 12 and v[0, 0, 0, 5, 19] == -2 and v[0, 0, 1, 14, 126] == -2 and v[0, 0, 1, 14, 127] == 1.5
    assert np.count_nonzero(v) == 4


def test_store_then_values():
    rng = np.random.default_rng(2)
    k, v = (rng.standard_normal((3, 2, 128)) * np.array([0.01, 1, 300])[:, None, None] for _ in range(2))
    v[1, 1, 37] = np.nan
    kv, scale, bits = ref.store_q4(np.full((2, 2, 2, 16, 64), 0x55, np.uint8), np.full((2, 2, 2, 128), 99, np.uint8), k, v, [17, -1, 3])
    got = ref.values_q4(kv, scale)
    assert bits == 0
    for row, (p, t) in ((0, (1, 1)), (2, (0, 3))):
        for w, x in ((0, k), (1, v)):
            g = x[row].reshape(2, 8, 16)
            step = np.abs(g).max(-1, keepdims=True) / 6 * 1.125  # at most half of the widest step, 2 scales, off
            assert (np.abs(got[p, :, w, t].reshape(2, 8, 16) - g) <= step).all()
    rest = np.ones(got.shape[:1] + (16,), bool)
    rest[1, 1] = rest[0, 3] = False
    assert (got[:, :, 0].swapaxes(1, 2)[rest] == ref.values_q4(np.full_like(kv, 0x55), np.full_like(scale, 99))[0, 0, 0, 0]).all()


def test_read_and_resume_by_hand():
    values = np.zeros((3, 1, 2, 16, 128))
    values[:] = np.arange(3 * 2 * 16).reshape(3, 1, 2, 16, 1)
    k, v, start, bits = ref.read(values, np.array([[2, 0], [1, -1]]), [18, 3], 30,
                                 (np.full((4, 1, 128), -1.0), np.full((4, 1, 128), -2.0), np.array([1, 2, 4])))
    assert start.tolist() == [0, 19, 24] and bits == 0
    assert k[:16, 0, 0].tolist() == list(range(64, 80)) and k[16:19, 0, 0].tolist() == [0, 1, -1]
    assert v[19:24, 0, 7].tolist() == [48, 49, 50, -2, -2] and np.isnan(k[24:]).all()
    k, v, start, bits = ref.read(values, np.array([[2, 0], [1, -1]]), [18, 3], 20)
    assert start.tolist() == [0, 18, 18] and bits == 8

    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((7, 2, 128)), rng.standard_normal((9, 1, 128)), rng.standard_normal((9, 1, 128))
    out, _, _, mine, bits = ref.resume(q, k, v, [0, 3, 3, 6, 7], [0, 5, 5, 8, 8], 0.1)
    assert bits == 8 and mine.tolist() == [True] * 6 + [False]  # the last one has no key
    whole = ref.prompt(np.concatenate([np.zeros((2, 2, 128)), q[:3]]), k[:5], v[:5], [0, 5], 0.1)[0]
    np.testing.assert_allclose(out[:3], whole[2:], rtol=1e-12)
    np.testing.assert_allclose(out[3:6], ref.prompt(q[3:6], k[5:8], v[5:8], [0, 3], 0.1)[0], rtol=1e-12)
