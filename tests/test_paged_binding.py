"""The binding's functions of the paged cache: every argument arrives where the header has the parameter of its name."""
import ctypes
import inspect
import os
import re

import numpy as np
import pytest

from sparse_decode_attention_oasis_gb300 import binding

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "oasis.h")
CALLS = ["oasis_extend_tables", "oasis_release_tables", "oasis_store_kv_q8", "oasis_store_kv_q4", "oasis_paged_decode_attn_q8",
         "oasis_paged_decode_attn_q4", "oasis_read_kv_q8", "oasis_read_kv_q4", "oasis_prompt_attn", "oasis_resume_attn",
         "oasis_resume_kv_q8", "oasis_resume_kv_q4"]
SIZES = ["oasis_paged_attn_workspace_bytes", "oasis_resume_attn_workspace_bytes", "oasis_resume_kv_workspace_bytes"]


def _parameters(name):
    """(type, name) of a function's parameters, from the header."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    (body,) = re.findall(r"OASIS_API\s+\w+\s+" + name + r"\s*\(([^)]*)\)", text)
    return [re.fullmatch(r"(.*?)\s*(\w+)", " ".join(p.split())).groups() for p in body.split(",")]


def _expected(ctype):
    return {"size_t": ctypes.c_size_t, "int32_t": ctypes.c_int32, "float": ctypes.c_float}.get(
        ctype, ctypes.POINTER(binding.PagedShape) if "oasis_paged_shape" in ctype else ctypes.c_void_p)


@pytest.mark.parametrize("name", CALLS + SIZES)
def test_arguments_in_the_headers_order(name, monkeypatch):
    class Recorder:
        def __getattr__(self, called):
            assert called == name
            return lambda *args: got.extend(args) or 0

    got = []
    monkeypatch.setattr(binding, "_lib", Recorder())
    header = _parameters(name)
    call = getattr(binding, name)
    mine = list(inspect.signature(call).parameters)
    assert [{"length": "len"}.get(n, n) for n in mine] == [n for _, n in header]
    values = {n: 1000 + i for i, n in enumerate(mine)}
    shape = values["shape"] = binding.PagedShape.of(2, 8, 2, 64, 100)
    call(**values)
    assert got[0]._obj is shape and got[1:] == list(values.values())[1:]


@pytest.mark.parametrize("name", CALLS + SIZES)
def test_types_of_the_headers_parameters(name):
    types, _ = binding._SIGS[name]
    want = [_expected(t) for t, _ in _parameters(name)]
    assert len(types) == len(want)
    for t, w in zip(types, want):
        assert t is w or (w is not ctypes.c_size_t and w not in (ctypes.c_int32, ctypes.c_float) and issubclass(t, (ctypes._Pointer, ctypes.c_void_p)))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_the_calls_on_a_gpu(bits):
    """Store, read-back, decode and resume through the binding against PagedKV's methods, bit by bit."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_helpers import bf16, ints

    from sparse_decode_attention_oasis_gb300 import binding as B
    from sparse_decode_attention_oasis_gb300.paged import PagedKV, resume_attn

    rng = np.random.default_rng(bits)
    hq, hkv, scale = 8, 2, 128 ** -0.5
    caches = [PagedKV(n_pages=40, batch=3, nb_max=12, n_q_heads=hq, n_kv_heads=hkv, bits=bits) for _ in range(2)]
    c, mine = caches
    for x in caches:
        x.kv.zero_()
        x.scale.fill_(1)
    rows = 70 + 33
    k, v = bf16(rng, (rows, hkv, 128))[0], bf16(rng, (rows, hkv, 128))[0]
    plan = c.extend(ints([70, 0, 33]), rows)
    mine.extend(ints([70, 0, 33]), rows)
    c.store(k, v, plan.slot_map)
    store, decode = getattr(B, f"oasis_store_kv_q{bits}"), getattr(B, f"oasis_paged_decode_attn_q{bits}")
    read, resume = getattr(B, f"oasis_read_kv_q{bits}"), getattr(B, f"oasis_resume_kv_q{bits}")
    shape, err = mine.shape, mine.err
    store(shape, k, hkv * 128, v, hkv * 128, plan.slot_map, rows, mine.kv, mine.scale, err)
    assert torch.equal(mine.kv, c.kv) and torch.equal(mine.scale, c.scale)

    q, _ = bf16(rng, (3, hq, 128))
    out = torch.empty_like(q)
    n = B.oasis_paged_attn_workspace_bytes(shape)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    decode(shape, q, hq * 128, mine.kv, mine.scale, c.table, plan.lens, None, None, 0, scale, ws, n, out, err)
    assert torch.equal(out, c.decode(q, plan.lens))

    new_start = ints([0, 4, 4, 9])
    want = c.read(rows + 9, plan.lens, new=(k[:9], v[:9], new_start), only_new=True)
    got_k, got_v = torch.zeros_like(want.k), torch.zeros_like(want.v)
    start = ints([0] * 4)
    read(shape, mine.kv, mine.scale, c.table, plan.lens, k, hkv * 128, v, hkv * 128, new_start, 9, 1, start, got_k, got_v, rows + 9, err)
    assert torch.equal(start, want.row_start)
    held = int(start[-1])
    assert torch.equal(got_k[:held], want.k[:held]) and torch.equal(got_v[:held], want.v[:held])

    q, _ = bf16(rng, (9, hq, 128))
    both = resume_attn(q, want.k[:held], want.v[:held], new_start, want.row_start)
    n = B.oasis_resume_attn_workspace_bytes(shape)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(q)
    B.oasis_resume_attn(shape, q, hq * 128, got_k, hkv * 128, got_v, hkv * 128, new_start, 9, start, held, scale, ws, n, out, hq * 128, err)
    assert torch.equal(out, both)
    n = B.oasis_resume_kv_workspace_bytes(shape, 9, rows)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros_like(q)
    resume(shape, q, hq * 128, k, hkv * 128, v, hkv * 128, new_start, 9, mine.kv, mine.scale, c.table, plan.lens, rows, scale, ws, n,
           out, hq * 128, err)
    assert torch.equal(out, both) and int(err) == 0
