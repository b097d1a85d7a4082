"""Shared pieces of the paged cache's tests: caches on the GPU beside oracle arrays, derived tolerances."""
import numpy as np

from oracle import paged_ref as ref

BF16_HALF_STEP = 2.0 ** -8  # torch.finfo(torch.bfloat16).eps / 2
F16_HALF_STEP = 2.0 ** -11


def bf16(rng, shape, size=1.0):
    """Normal values on the GPU in bf16, and the same in 64 bits."""
    import torch

    t = torch.from_numpy((rng.standard_normal(shape) * size).astype(np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def ints(values):
    import torch

    return torch.tensor(np.asarray(values), dtype=torch.int32).cuda()


def random_pages(rng, n_pages, hkv, low=-9, high=-5):
    """Bytes of normal values (no NaN), and power-of-two scales that differ from page to page."""
    kv = ref.e4m3_bytes(rng.standard_normal((n_pages, hkv, 2, 16, 128)) * 60.0)
    return kv, 2.0 ** rng.integers(low, high, (n_pages, hkv, 2)).astype(np.float64)


def shuffled_table(rng, ctx, nb_max, n_pages):
    table = np.full((len(ctx), nb_max), -1)
    order, at = rng.permutation(n_pages), 0
    for b, n in enumerate(ctx):
        nb = min(-(-max(n, 0) // 16), nb_max)
        table[b, :nb] = order[at:at + nb]
        at += nb
    assert at <= n_pages
    return table


def cache_of(kv, scale, table, hq):
    import torch

    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    c = PagedKV(n_pages=kv.shape[0], batch=table.shape[0], nb_max=table.shape[1], n_q_heads=hq, n_kv_heads=kv.shape[1])
    c.kv[0] = torch.from_numpy(kv).cuda()
    c.scale[0] = torch.from_numpy(scale.astype(np.float32)).cuda()
    c.table.copy_(ints(table))
    return c


def check_attention(got, want, mass, size, weight_step, tiny=0.0):
    """|got - want| against what the roundings allow, element by element:
      the output's rounding                    2^-8 |out|
      the weights' rounding for the product    weight_step * sum p |v|
      scores in fp32: 128 products accumulated on tensor cores with at most 2^-15.9 |q||k| of
      error, scale and exponent rounded a few times (2^-22 of the score); a relative weight
      error of d changes numerator and denominator: 2 d sum p |v|
      fp32 accumulation of weights and products  2^-15 sum p |v| (thousands of truncated steps)
      fp16 weights below its normal range        2^-25 max|v| tokens / sum, given as `tiny`"""
    d = size * (2.0 ** -15.9 + 2.0 ** -21)
    tol = BF16_HALF_STEP * np.abs(want) + (weight_step + 2 * d + 2.0 ** -15) * mass + 2.0 ** -25 * tiny + 1e-30
    # the output's rounding is of the computed value
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol * (1 + BF16_HALF_STEP)).all(), f"{int((err > tol).sum())} elements, worst {np.max(err / tol):.2f} x allowed"
