"""Refusals of the paged cache's calls: all before any launch, so no GPU is needed."""
import ctypes

import pytest

from sparse_decode_attention_oasis_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _shape(**kw):
    base = dict(B=2, Hq=32, Hkv=8, nb_max=64, n_pages=100)
    base.update(kw)
    return binding.PagedShape.of(**base)


SHAPES = [(dict(Hq=30), 1), (dict(B=0), 1), (dict(n_pages=0), 1), (dict(nb_max=-1), 1), (dict(d=64), 4), (dict(bs=32), 4),
          (dict(Hq=72), 4), (dict(B=65536), 4), (dict(Hq=1025, Hkv=1025), 4), (dict(B=65535, Hq=32, Hkv=32), 4),
          (dict(nb_max=(1 << 24) + 1), 4), (dict(n_pages=1 << 27), 4)]


def _prompt(lib, s, q=16, qs=4096, k=16, ks=1024, v=16, vs=1024, start=16, n=5, scale=0.1, out=16, os=4096, err=None):
    return lib.oasis_prompt_attn(ctypes.byref(s), q, qs, k, ks, v, vs, start, n, scale, out, os, err, None)


def _decode(lib, s, q=16, qs=4096, kv=16, sc=16, table=16, ctx=16, sel=None, nsel=None, most=0, scale=0.1, ws=16,
            nb=1 << 30, out=16, err=None):
    return lib.oasis_paged_decode_attn_q8(ctypes.byref(s), q, qs, kv, sc, table, ctx, sel, nsel, most, scale, ws, nb,
                                          out, err, None)


def _store(lib, s, k=16, ks=1024, v=16, vs=1024, slots=16, n=5, kv=16, sc=16, err=None):
    return lib.oasis_store_kv_q8(ctypes.byref(s), k, ks, v, vs, slots, n, kv, sc, err, None)


def _extend(lib, s, old=1024, new=2048, free=16, nf=4096, table=16, lens=8192, nfo=12288, start=16, slots=16, n=5,
            err=None):
    return lib.oasis_extend_tables(ctypes.byref(s), old, new, free, nf, table, lens, nfo, start, slots, n, err, None)


def _release(lib, s, length=16, keep=16, table=16, free=16, nf=16, nfo=32, err=None):
    return lib.oasis_release_tables(ctypes.byref(s), length, keep, table, free, nf, nfo, err, None)


@pytest.mark.parametrize("kw,status", SHAPES)
def test_every_call_checks_the_shape(lib, kw, status):
    s = _shape(**kw)
    for call in (_prompt, _decode, _store, _extend, _release):
        assert call(lib, s) == status, call.__name__
        assert lib.oasis_last_error().startswith(b"oasis_")
    assert lib.oasis_paged_attn_workspace_bytes(ctypes.byref(s)) == 0


def test_a_missing_shape_is_invalid(lib):
    assert lib.oasis_prompt_attn(None, 16, 4096, 16, 1024, 16, 1024, 16, 5, 0.1, 16, 4096, None, None) == 1
    assert lib.oasis_paged_attn_workspace_bytes(None) == 0


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=8), dict(qs=4095), dict(qs=4088), dict(qs=1 << 32), dict(k=None), dict(ks=1020), dict(ks=1016),
    dict(v=24), dict(vs=0), dict(start=None), dict(start=18), dict(n=-1), dict(n=(1 << 26) + 1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(out=None), dict(out=8), dict(os=4088), dict(err=2)])
def test_prompt_refusals(lib, kw):
    assert _prompt(lib, _shape(), **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=8), dict(qs=4088), dict(qs=4097), dict(kv=None), dict(kv=8), dict(sc=None), dict(sc=4),
    dict(table=None), dict(ctx=None), dict(ctx=2), dict(sel=16), dict(nsel=16), dict(sel=16, nsel=16, most=0),
    dict(sel=16, nsel=16, most=65537), dict(sel=18, nsel=16, most=4), dict(scale=0.0), dict(scale=NAN), dict(scale=INF),
    dict(ws=None), dict(ws=8), dict(nb=16), dict(out=None), dict(out=8), dict(err=1)])
def test_decode_refusals(lib, kw):
    assert _decode(lib, _shape(), **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(k=8), dict(ks=1016), dict(ks=1025), dict(v=None), dict(vs=8), dict(slots=None), dict(slots=2),
    dict(n=-1), dict(kv=None), dict(kv=8), dict(sc=4), dict(sc=None), dict(err=3)])
def test_store_refusals(lib, kw):
    assert _store(lib, _shape(), **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(old=None), dict(new=2), dict(free=None), dict(nf=None), dict(table=None), dict(lens=None), dict(nfo=None),
    dict(start=None), dict(slots=None), dict(n=-1), dict(n=(1 << 28) + 1), dict(err=2),
    dict(lens=1024), dict(lens=1028), dict(lens=2044), dict(nfo=4096), dict(nfo=1028), dict(lens=4092)])
def test_extend_refusals(lib, kw):
    assert _extend(lib, _shape(), **kw) == 1


@pytest.mark.parametrize("kw", [dict(length=None), dict(keep=2), dict(table=None), dict(free=None), dict(nf=None),
                                dict(nfo=None), dict(nfo=16), dict(err=2)])
def test_release_refusals(lib, kw):
    assert _release(lib, _shape(), **kw) == 1


def test_nothing_to_do_needs_no_rows(lib):
    s = _shape()
    assert _prompt(lib, s, q=None, k=None, v=None, out=None, n=0) == 0
    assert _store(lib, s, k=None, v=None, slots=None, n=0) == 0


def test_workspace_does_not_depend_on_the_context(lib):
    a, b = _shape(nb_max=1), _shape(nb_max=1 << 20, n_pages=1 << 20, B=500)
    n = lib.oasis_paged_attn_workspace_bytes(ctypes.byref(a))
    assert n == lib.oasis_paged_attn_workspace_bytes(ctypes.byref(b)) > 0


def test_python_layer_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    from sparse_decode_attention_oasis_gb300.paged import prompt_attn

    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        prompt_attn(q, q[:, :1], q[:, :1], torch.zeros(2, dtype=torch.int32))
