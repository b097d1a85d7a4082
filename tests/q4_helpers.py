"""Shared pieces of the 4-bit cache's tests: pages, tables and caches on the GPU beside oracle arrays."""
import numpy as np

from oracle import paged_ref as ref


def random_pages_q4(rng, n_pages, hkv, low=12, high=14):
    """Random codes, and scale bytes with exponent fields low .. high - 1."""
    kv = rng.integers(0, 256, (n_pages, hkv, 2, 16, 64)).astype(np.uint8)
    return kv, rng.integers(low * 8, high * 8, (n_pages, hkv, 2, 128)).astype(np.uint8)


def cache_q4(kv, scale, table, hq):
    import torch

    from paged_helpers import ints
    from sparse_decode_attention_oasis_gb300.paged import PagedKV

    c = PagedKV(n_pages=kv.shape[0], batch=table.shape[0], nb_max=table.shape[1], n_q_heads=hq, n_kv_heads=kv.shape[1], bits=4)
    c.kv[0] = torch.from_numpy(kv).cuda()
    c.scale[0] = torch.from_numpy(scale).cuda()
    c.table.copy_(ints(table))
    return c


def pages_and_cache(bits, rng, n_pages, hkv, hq, table):
    """(values in 64 bits, cache) of random pages in 8 or 4 bits."""
    from paged_helpers import cache_of, random_pages

    if bits == 8:
        kv, scale = random_pages(rng, n_pages, hkv)
        return ref.E4M3[kv] * scale[..., None, None], cache_of(kv, scale, table, hq)
    kv, scale = random_pages_q4(rng, n_pages, hkv)
    return ref.values_q4(kv, scale), cache_q4(kv, scale, table, hq)
