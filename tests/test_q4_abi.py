"""Refusals of the 4-bit cache's calls, of the read-back and of the resumed attention: all before any launch."""
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


def _store(lib, s, k=16, ks=1024, v=16, vs=1024, slots=16, n=5, kv=16, sc=16, err=None):
    return lib.oasis_store_kv_q4(ctypes.byref(s), k, ks, v, vs, slots, n, kv, sc, err, None)


def _decode(lib, s, q=16, qs=4096, kv=16, sc=16, table=16, ctx=16, sel=None, nsel=None, most=0, scale=0.1, ws=16,
            nb=1 << 30, out=16, err=None):
    return lib.oasis_paged_decode_attn_q4(ctypes.byref(s), q, qs, kv, sc, table, ctx, sel, nsel, most, scale, ws, nb,
                                          out, err, None)


def _read(lib, s, kv=16, sc=16, table=16, ctx=16, k=16, ks=1024, v=16, vs=1024, new=16, n_new=3, only=0, start=16, ko=32, vo=32,
          n=5, err=None, bits=4):
    call = lib.oasis_read_kv_q4 if bits == 4 else lib.oasis_read_kv_q8
    return call(ctypes.byref(s), kv, sc, table, ctx, k, ks, v, vs, new, n_new, only, start, ko, vo, n, err, None)


def _resume(lib, s, q=16, qs=4096, k=16, ks=1024, v=16, vs=1024, start=16, n=5, kstart=16, m=9, scale=0.1, ws=32, nb=1 << 30,
            out=16, os=4096, err=None):
    return lib.oasis_resume_attn(ctypes.byref(s), q, qs, k, ks, v, vs, start, n, kstart, m, scale, ws, nb, out, os, err, None)


def _resume_kv(lib, s, q=16, qs=4096, k=16, ks=1024, v=16, vs=1024, start=16, n=50, kv=16, sc=16, table=16, ctx=16, held=9, scale=0.1,
               ws=32, nb=1 << 30, out=16, os=4096, err=None, bits=4):
    call = lib.oasis_resume_kv_q4 if bits == 4 else lib.oasis_resume_kv_q8
    return call(ctypes.byref(s), q, qs, k, ks, v, vs, start, n, kv, sc, table, ctx, held, scale, ws, nb, out, os, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=30), 1), (dict(B=0), 1), (dict(n_pages=0), 1), (dict(d=64), 4), (dict(bs=32), 4), (dict(Hq=72), 4),
    (dict(B=65536), 4), (dict(nb_max=(1 << 24) + 1), 4), (dict(n_pages=1 << 27), 4)])
def test_every_call_checks_the_shape(lib, kw, status):
    s = _shape(**kw)
    for call in (_store, _decode, _read, _resume):
        assert call(lib, s) == status, call.__name__
        assert lib.oasis_last_error().startswith(b"oasis_")
    assert _read(lib, s, bits=8) == status
    assert lib.oasis_resume_attn_workspace_bytes(ctypes.byref(s)) == 0
    assert lib.oasis_resume_attn_workspace_bytes(None) == 0


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(k=8), dict(ks=1016), dict(ks=1025), dict(v=None), dict(vs=8), dict(slots=None), dict(slots=2),
    dict(n=-1), dict(n=(1 << 28) + 1), dict(kv=None), dict(kv=8), dict(sc=8), dict(sc=None), dict(err=3)])
def test_store_refusals(lib, kw):
    assert _store(lib, _shape(), **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=8), dict(qs=4088), dict(qs=4097), dict(kv=None), dict(kv=8), dict(sc=None), dict(sc=8),
    dict(table=None), dict(ctx=None), dict(ctx=2), dict(sel=16), dict(nsel=16), dict(sel=16, nsel=16, most=0),
    dict(sel=16, nsel=16, most=65537), dict(scale=0.0), dict(scale=NAN), dict(scale=INF), dict(ws=None), dict(ws=8), dict(nb=16),
    dict(out=None), dict(out=8), dict(err=1)])
def test_decode_refusals(lib, kw):
    assert _decode(lib, _shape(), **kw) == 1


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kw", [
    dict(kv=None), dict(kv=8), dict(sc=None), dict(sc=4), dict(table=None), dict(ctx=2), dict(start=None), dict(start=2),
    dict(k=None), dict(k=8), dict(ks=1016), dict(vs=1028), dict(v=None), dict(new=2), dict(n_new=-1), dict(n_new=(1 << 28) + 1),
    dict(n=-1), dict(n=(1 << 28) + 1), dict(ko=None), dict(ko=16), dict(vo=48), dict(err=2)])
def test_read_refusals(lib, bits, kw):
    assert _read(lib, _shape(), bits=bits, **kw) == 1


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=8), dict(qs=4095), dict(qs=4088), dict(qs=1 << 32), dict(k=None), dict(ks=1020), dict(v=24), dict(vs=0),
    dict(start=None), dict(start=18), dict(kstart=None), dict(kstart=2), dict(n=-1), dict(n=(1 << 26) + 1), dict(m=-1), dict(m=0),
    dict(m=(1 << 26) + 1), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(ws=None), dict(ws=16),
    dict(nb=16), dict(out=None), dict(out=8), dict(os=4088), dict(err=2)])
def test_resume_refusals(lib, kw):
    assert _resume(lib, _shape(), **kw) == 1


def test_nothing_to_do_needs_no_rows(lib):
    s = _shape()
    assert _store(lib, s, k=None, v=None, slots=None, n=0) == 0
    assert _resume(lib, s, q=None, k=None, v=None, out=None, ws=None, nb=0, n=0, m=0) == 0


def test_the_resumes_workspace_does_not_depend_on_the_sizes(lib):
    a, b = _shape(nb_max=1, B=1, Hq=1, Hkv=1), _shape(nb_max=1 << 20, B=500, Hq=64)
    n = lib.oasis_resume_attn_workspace_bytes(ctypes.byref(a))
    assert n == lib.oasis_resume_attn_workspace_bytes(ctypes.byref(b)) > 0


def test_the_python_layer_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    from sparse_decode_attention_oasis_gb300.paged import resume_attn

    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    start = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        resume_attn(q, q[:, :1], q[:, :1], start, start)


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=30), 1), (dict(B=0), 1), (dict(n_pages=0), 1), (dict(d=64), 4), (dict(bs=32), 4), (dict(Hq=72), 4),
    (dict(B=65536), 4), (dict(nb_max=(1 << 24) + 1), 4), (dict(n_pages=1 << 27), 4)])
def test_resume_over_pages_checks_the_shape(lib, kw, status):
    s = _shape(**kw)
    assert _resume_kv(lib, s) == _resume_kv(lib, s, bits=8) == status
    assert lib.oasis_last_error().startswith(b"oasis_resume_kv_q8")
    assert lib.oasis_resume_kv_workspace_bytes(ctypes.byref(s), 5, 5) == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=8), dict(qs=4095), dict(k=None), dict(ks=1020), dict(v=24), dict(vs=0), dict(start=None), dict(start=18),
    dict(n=-1), dict(n=(1 << 26) + 1), dict(held=-1), dict(held=(1 << 26) + 1), dict(kv=None), dict(kv=8), dict(sc=None), dict(sc=4),
    dict(table=None), dict(table=2), dict(ctx=None), dict(scale=0.0), dict(scale=NAN), dict(ws=None), dict(ws=16), dict(nb=16),
    dict(out=None), dict(out=8), dict(os=4088), dict(err=2)])
def test_resume_over_pages_refusals(lib, bits, kw):
    assert _resume_kv(lib, _shape(), bits=bits, **kw) == 1


def test_the_workspace_over_pages(lib):
    s = ctypes.byref(_shape())
    none = lib.oasis_resume_kv_workspace_bytes(s, 0, 0)
    assert none >= lib.oasis_resume_attn_workspace_bytes(s) > 0
    assert lib.oasis_resume_kv_workspace_bytes(s, 33, 1000) == none + 1033 * 4 * 8 * 128
    for n, held in ((-1, 0), (0, -1), (1 << 26, 1)):
        assert lib.oasis_resume_kv_workspace_bytes(s, n, held) == 0
    assert _resume_kv(lib, _shape(), n=50, held=9, nb=none + 59 * 4 * 8 * 128 - 1) == 1
    assert _resume_kv(lib, _shape(), q=None, k=None, v=None, out=None, ws=None, nb=0, n=0) == 0  # nothing to do
