"""A KV cache in 8-bit or 4-bit pages: tables, store, decode attention, read-back, and the prompts' attention.

PyTorch owns the memory and the streams; every step runs in liboasis.so through
:mod:`binding`.  One :class:`PagedKV` serves a model of several layers whose requests
share the tables:

  kv     uint8   [layers][n_pages][Hkv][2][16][128]   e4m3 keys, values
  scale  float32 [layers][n_pages][Hkv][2]            powers of two
  with bits=4:
  kv     uint8   [layers][n_pages][Hkv][2][16][64]    e2m1 keys, values, two to a byte
  scale  uint8   [layers][n_pages][Hkv][2][128]       for 16 dimensions of a token
  table  int32   [batch][nb_max]                      page of each request's blocks
  free   int32   [n_pages]                            free pages, the first n_free of them
  lens   int32   [batch]                              tokens that each request holds
  err    int32   [1]                                  error word (OASIS_EW_* bits)

A prompt's pass, layer by layer, and a decode step::

    plan = cache.extend(lens, n_rows)                  # pages and slots of the new tokens
    out = cache.prompt(q, k, v, plan)                  # requests that held nothing before
    cache.store(k, v, plan.slot_map, layer)
    cache.commit(plan)
    cache.check()                                      # raises what the kernels reported
    ...
    plan = cache.extend(cache.lens + 1, batch)
    cache.store(k, v, plan.slot_map, layer)
    out = cache.decode(q, plan.lens, layer)            # sel, nsel: only the selected blocks
    cache.commit(plan)

A prompt that continues a context attends what its request holds as well as itself::

    plan = cache.extend(cache.lens + more, n_rows)     # held: at least the tokens that these requests hold in all
    out = cache.resume(q, k, v, plan, held, layer)     # before commit
    cache.store(k, v, plan.slot_map, layer)
    cache.commit(plan)

Calls run on the current stream of the tensors' device and can be captured into a CUDA
graph; nothing is kept between calls but the tensors above and the scratch of decode and of resume,
one for each stream (calls on one stream follow each other, those of several host threads as well:
the library keeps a call's launches together; resume keeps at most 256 MB, and takes more from PyTorch's memory for
the call alone).  A captured call takes scratch of its
own from the graph's memory pool, so graphs, and calls on other streams, never share it.

The methods call the library directly with addresses and sizes: for a decode step's small
kernels the host's share of a call is what counts.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple, Optional

import torch

from . import binding as B

D = 128
BS = 16
_SCALE = 1.0 / math.sqrt(D)
_BF16, _INT32 = torch.bfloat16, torch.int32
_KEPT = 256 << 20  # bytes of resume's scratch that stay (allocated at each call, a short one takes 17.5 us, else 12.8)


class Rows(NamedTuple):
    """What :meth:`PagedKV.read` gives: request b's tokens are rows row_start[b] .. row_start[b+1] - 1."""

    k: torch.Tensor          # bfloat16 [n_rows][Hkv][128]
    v: torch.Tensor
    row_start: torch.Tensor  # int32 [batch + 1]


class Plan(NamedTuple):
    """What :meth:`PagedKV.extend` gives: it takes effect with :meth:`PagedKV.commit`."""

    lens: torch.Tensor       # int32 [batch]: lengths that the tables now hold
    n_free: torch.Tensor     # int32 [1]
    row_start: torch.Tensor  # int32 [batch + 1]: first new row of each request
    slot_map: torch.Tensor   # int32 [n_rows]: page * 16 + position, -1 for rows of no request


_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _cuda(device: torch.device) -> int:
    if device.type != "cuda":
        raise ValueError("CUDA tensors are needed (there is no CPU path)")
    return device.index


def _rows(name: str, t: torch.Tensor, heads: int, n: int, device) -> int:
    """Checks bf16 rows [n][heads][128], contiguous inside a row; returns the row stride."""
    if t.dtype is not _BF16 or t.shape != (n, heads, D) or t.device != device:
        raise ValueError(f"{name} must be bfloat16 [{n}, {heads}, {D}] on {device}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    if n == 0:
        return heads * D
    stride, inner, one = t.stride()
    if n == 1:
        stride = heads * D
    if one != 1 or (inner != D and heads > 1) or stride < heads * D or stride % 8:
        raise ValueError(f"{name}: a row's heads and dimensions must be contiguous, rows a multiple of 8 elements "
                         f"and at least {heads * D} apart (strides {t.stride()})")
    return stride


def _ints(name: str, t: torch.Tensor, shape, device) -> torch.Tensor:
    if t.dtype is not _INT32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")
    return t


@functools.lru_cache(maxsize=256)
def _prompt_shape(sequences: int, hq: int, hkv: int):
    return ctypes.byref(B.PagedShape(sequences, hq, hkv, D, BS, 1, 1))


@functools.lru_cache(maxsize=256)
def _resume_bytes(sequences: int, hq: int, hkv: int, index: int) -> int:
    n = (B._lib or B.load()).oasis_resume_attn_workspace_bytes(_prompt_shape(sequences, hq, hkv))
    if not n:
        raise B.OasisError("oasis_resume_attn_workspace_bytes", 1, B.oasis_last_error())
    return n


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, row_start: torch.Tensor,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention over packed prompts: q [rows, Hq, 128], k and v [rows, Hkv, 128] in
    bf16 (slices of one buffer as well), sequence b in rows row_start[b] .. row_start[b+1] - 1.
    Rows of no sequence are left as they are in out (zero where out is allocated here).

    A row attends the call's own rows of its sequence and nothing that a cache holds.  Errors
    (a bad row_start, a wait inside the kernel that gave up: incomplete output) go to err and
    nowhere else; :meth:`PagedKV.prompt` passes the cache's."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [rows, heads, 128]")
    n, hq, hkv, device = q.shape[0], q.shape[1], k.shape[1], q.device
    index = _cuda(device)
    if _current_device() != index:
        with torch.cuda.device(index):
            return prompt_attn(q, k, v, row_start, scale, out, err)
    qs, ks, vs = _rows("q", q, hq, n, device), _rows("k", k, hkv, n, device), _rows("v", v, hkv, n, device)
    sequences = row_start.numel() - 1
    if sequences < 1:
        raise ValueError("row_start must be int32 [sequences + 1]")
    _ints("row_start", row_start, (sequences + 1,), device)
    if out is None:
        out = torch.zeros((n, hq, D), dtype=_BF16, device=device)
    st = (B._lib or B.load()).oasis_prompt_attn(
        _prompt_shape(sequences, hq, hkv), q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, row_start.data_ptr(), n,
        _SCALE if scale is None else scale, out.data_ptr(), _rows("out", out, hq, n, device),
        None if err is None else _ints("err", err, (1,), device).data_ptr(), _current_stream(index))
    if st:
        B._check("oasis_prompt_attn", st)
    return out


def resume_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, kv_start: torch.Tensor,
                scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Causal attention of new rows that continue a context: q [rows, Hq, 128] in rows q_start[b] ..
    q_start[b+1] - 1 for sequence b, k and v [kv_rows, Hkv, 128] in rows kv_start[b] .. kv_start[b+1] - 1, its
    earlier tokens first and then one for each of its query rows (bf16; slices of one buffer as well).
    Rows of no sequence are left as they are in out (zero where out is allocated here).

    Errors (bad starts, fewer rows of keys than of queries, a wait inside the kernel that gave up) go
    to err and nowhere else; :meth:`PagedKV.resume` passes the cache's."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [rows, heads, 128]")
    n, hq, m, hkv, device = q.shape[0], q.shape[1], k.shape[0], k.shape[1], q.device
    index = _cuda(device)
    if _current_device() != index:
        with torch.cuda.device(index):
            return resume_attn(q, k, v, q_start, kv_start, scale, out, err)
    qs, ks, vs = _rows("q", q, hq, n, device), _rows("k", k, hkv, m, device), _rows("v", v, hkv, m, device)
    sequences = q_start.numel() - 1
    if sequences < 1:
        raise ValueError("q_start must be int32 [sequences + 1]")
    _ints("q_start", q_start, (sequences + 1,), device)
    _ints("kv_start", kv_start, (sequences + 1,), device)
    if out is None:
        out = torch.zeros((n, hq, D), dtype=_BF16, device=device)
    shape = _prompt_shape(sequences, hq, hkv)
    ws_bytes = _resume_bytes(sequences, hq, hkv, index)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
    st = (B._lib or B.load()).oasis_resume_attn(
        shape, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, q_start.data_ptr(), n, kv_start.data_ptr(), m,
        _SCALE if scale is None else scale, ws.data_ptr(), ws_bytes, out.data_ptr(), _rows("out", out, hq, n, device),
        None if err is None else _ints("err", err, (1,), device).data_ptr(), _current_stream(index))
    if st:
        B._check("oasis_resume_attn", st)
    return out


class PagedKV:
    def __init__(self, n_pages: int, batch: int, nb_max: int, n_q_heads: int, n_kv_heads: int, layers: int = 1,
                 device="cuda", bits: int = 8):
        if bits not in (4, 8):
            raise ValueError(f"pages hold 4 or 8 bits, not {bits}")
        self.bits = bits
        self.shape = B.PagedShape.of(batch, n_q_heads, n_kv_heads, nb_max, n_pages)
        self.ws_bytes = B.oasis_paged_attn_workspace_bytes(self.shape)  # also checks the shape
        if not self.ws_bytes:
            raise B.OasisError("oasis_paged_attn_workspace_bytes", 1, B.oasis_last_error())
        if layers < 1:
            raise ValueError("layers must be >= 1")
        self.batch, self.n_q_heads, self.n_kv_heads, self.layers = batch, n_q_heads, n_kv_heads, layers
        # not initialised: positions that were never stored are never read
        self.kv = torch.empty((layers, n_pages, n_kv_heads, 2, BS, D * bits // 8), dtype=torch.uint8, device=device)
        if bits == 8:
            self.scale = torch.ones((layers, n_pages, n_kv_heads, 2), dtype=torch.float32, device=device)
        else:
            self.scale = torch.empty((layers, n_pages, n_kv_heads, 2, BS * D // 16), dtype=torch.uint8, device=device)
        self.table = torch.full((batch, nb_max), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)  # page 0 is taken first
        self.n_free = torch.full((1,), n_pages, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = self.kv.device
        self._index = _cuda(self.device)
        self._shape = ctypes.byref(self.shape)
        self._kv_bytes, self._scale_bytes = self.kv.stride(0), self.scale.element_size() * self.scale.stride(0)  # of a layer
        self._scratch, self._resume_scratch = {}, {}  # decode's, resume's, by stream
        with torch.cuda.device(self._index):  # resume's scratch, and 4 * Hkv * 128 for each row and held token
            self._resume_bytes = B.oasis_resume_kv_workspace_bytes(self.shape, 0, 0)

    def adopt(self, **tensors: torch.Tensor) -> None:
        """Use the caller's tensors in place of kv, scale, table, free, n_free or lens (same
        shape, type and device): a pool that the program owns already, or a saved state."""
        for name, t in tensors.items():
            if name not in ("kv", "scale", "table", "free", "n_free", "lens"):
                raise ValueError(f"no tensor {name}")
            mine = getattr(self, name)
            if t.dtype != mine.dtype or t.shape != mine.shape or t.device != mine.device or not t.is_contiguous() \
                    or t.data_ptr() % 16:
                raise ValueError(f"{name} must be contiguous, 16-byte aligned {mine.dtype} {tuple(mine.shape)} on "
                                 f"{mine.device}")
        for name, t in tensors.items():
            setattr(self, name, t)

    def extend(self, new_len: torch.Tensor, n_rows: int) -> Plan:
        """Pages for requests that grow to new_len tokens and slots for their new rows (at most
        n_rows).  Only new table entries are written: lens and n_free change with commit."""
        b = self.batch
        device = self.device
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.extend(new_len, n_rows)
        _ints("new_len", new_len, (b,), device)
        if n_rows < 0:
            raise ValueError("n_rows must be >= 0")
        # four allocations: views of one cost more on the host than the launch
        lens, n_free = torch.empty_like(self.lens), torch.empty_like(self.n_free)
        row_start = torch.empty(b + 1, dtype=_INT32, device=device)
        slot_map = torch.empty(n_rows, dtype=_INT32, device=device)
        st = (B._lib or B.load()).oasis_extend_tables(
            self._shape, self.lens.data_ptr(), new_len.data_ptr(), self.free.data_ptr(), self.n_free.data_ptr(),
            self.table.data_ptr(), lens.data_ptr(), n_free.data_ptr(), row_start.data_ptr(), slot_map.data_ptr(), n_rows,
            self.err.data_ptr(), _current_stream(self._index))
        if st:
            B._check("oasis_extend_tables", st)
        return Plan(lens, n_free, row_start, slot_map)

    def commit(self, plan: Plan) -> None:
        """The plan's lengths and free count become the cache's."""
        self.lens.copy_(plan.lens)
        self.n_free.copy_(plan.n_free)

    def release(self, keep_len: torch.Tensor) -> None:
        """Requests keep their first keep_len tokens (0: the request is done); the pages of the
        others are free again."""
        _ints("keep_len", keep_len, (self.batch,), self.device)
        with torch.cuda.device(self._index):
            left = torch.empty_like(self.n_free)
            B.oasis_release_tables(self.shape, self.lens, keep_len, self.table, self.free, self.n_free, left, self.err)
            self.n_free.copy_(left)
            kept = (keep_len >= 0) & (keep_len <= self.lens)  # the others released nothing
            self.lens.copy_(torch.where(kept, keep_len, self.lens))

    def prompt(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: Plan, scale: Optional[float] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """:func:`prompt_attn` over a plan's rows; :meth:`check` raises its errors.  For plans whose
        new rows are all of requests that held nothing before: earlier tokens are not attended (:meth:`resume`
        attends them)."""
        if q.dim() != 3 or q.shape[1] != self.n_q_heads or k.dim() != 3 or k.shape[1] != self.n_kv_heads:
            raise ValueError(f"q must be [rows, {self.n_q_heads}, 128], k and v [rows, {self.n_kv_heads}, 128]")
        return prompt_attn(q, k, v, plan.row_start, scale, out, self.err)

    def store(self, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, layer: int = 0) -> None:
        """Rows k, v [rows, Hkv, 128] (bf16) into the layer's pages at slot_map's slots."""
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.store(k, v, slot_map, layer)
        n, h, device = slot_map.numel(), self.n_kv_heads, self.device
        ks, vs = _rows("k", k, h, n, device), _rows("v", v, h, n, device)
        _ints("slot_map", slot_map, (n,), device)
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of {self.layers}")
        lib = B._lib or B.load()
        st = (lib.oasis_store_kv_q8 if self.bits == 8 else lib.oasis_store_kv_q4)(
            self._shape, k.data_ptr(), ks, v.data_ptr(), vs, slot_map.data_ptr(), n,
            self.kv.data_ptr() + layer * self._kv_bytes, self.scale.data_ptr() + layer * self._scale_bytes,
            self.err.data_ptr(), _current_stream(self._index))
        if st:
            B._check(f"oasis_store_kv_q{self.bits}", st)

    def decode(self, q: torch.Tensor, ctx_len: Optional[torch.Tensor] = None, layer: int = 0,
               sel: Optional[torch.Tensor] = None, nsel: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of q [batch, Hq, 128] (bf16) over the first ctx_len tokens of every request
        (lens by default), or over the blocks that sel [batch, Hkv, most], nsel [batch, Hkv] list."""
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.decode(q, ctx_len, layer, sel, nsel, scale, out)
        b, hq, device = self.batch, self.n_q_heads, self.device
        stride = _rows("q", q, hq, b, device)
        ctx_len = _ints("ctx_len", self.lens if ctx_len is None else ctx_len, (b,), device)
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of {self.layers}")
        most, sel_at, nsel_at = 0, None, None
        if sel is not None or nsel is not None:
            if sel is None or nsel is None or sel.dim() != 3:
                raise ValueError("sel [batch, Hkv, most] and nsel [batch, Hkv] must be given together")
            most = sel.shape[2]
            sel_at = _ints("sel", sel, (b, self.n_kv_heads, most), device).data_ptr()
            nsel_at = _ints("nsel", nsel, (b, self.n_kv_heads), device).data_ptr()
        if out is None:
            out = torch.empty((b, hq, D), dtype=_BF16, device=device)
        elif out.dtype is not _BF16 or out.shape != (b, hq, D) or out.device != device or not out.is_contiguous():
            raise ValueError(f"out must be contiguous bfloat16 [{b}, {hq}, {D}] on {device}")
        stream = _current_stream(self._index)
        capturing = torch._C._cuda_isCurrentStreamCapturing()
        ws = None if capturing else self._scratch.get(stream)
        if ws is None:
            ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
            if not capturing:
                self._scratch[stream] = ws
        lib = B._lib or B.load()
        st = (lib.oasis_paged_decode_attn_q8 if self.bits == 8 else lib.oasis_paged_decode_attn_q4)(
            self._shape, q.data_ptr(), stride, self.kv.data_ptr() + layer * self._kv_bytes,
            self.scale.data_ptr() + layer * self._scale_bytes, self.table.data_ptr(), ctx_len.data_ptr(), sel_at, nsel_at,
            most, _SCALE if scale is None else scale, ws.data_ptr(), self.ws_bytes, out.data_ptr(), self.err.data_ptr(),
            stream)
        if st:
            B._check(f"oasis_paged_decode_attn_q{self.bits}", st)
        return out

    def read(self, n_rows: int, ctx_len: Optional[torch.Tensor] = None, layer: int = 0, new=None, out=None,
             only_new: bool = False) -> Rows:
        """The first ctx_len tokens of every request (lens by default) as packed bf16 rows, at most n_rows
        of them; stored values are bf16 exactly.  new = (k, v, row_start) puts the rows row_start[b] ..
        row_start[b+1] - 1 of k and v [rows, Hkv, 128] behind request b's; with only_new requests without new
        rows have no rows at all.  out = (k, v): contiguous bf16
        [n_rows, Hkv, 128] to write to, or (k, v, row_start) with int32 [batch + 1] as well (an earlier call's Rows),
        none of which lies on what the call reads; rows behind the last request's are left as they are."""
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.read(n_rows, ctx_len, layer, new, out, only_new)
        b, h, device = self.batch, self.n_kv_heads, self.device
        ctx_len = _ints("ctx_len", self.lens if ctx_len is None else ctx_len, (b,), device)
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of {self.layers}")
        if n_rows < 0:
            raise ValueError("n_rows must be >= 0")
        k_at = v_at = ks = vs = n_new = 0
        start_at = None
        if new is not None:
            k, v, row_start = new
            if k.dim() != 3:
                raise ValueError("new rows must be [rows, heads, 128]")
            n_new = k.shape[0]
            ks, vs = _rows("k", k, h, n_new, device), _rows("v", v, h, n_new, device)
            k_at, v_at = k.data_ptr(), v.data_ptr()
            start_at = _ints("row_start", row_start, (b + 1,), device).data_ptr()
        kv_start = None
        if out is None:
            out = (torch.empty((n_rows, h, D), dtype=_BF16, device=device), torch.empty((n_rows, h, D), dtype=_BF16, device=device))
        else:
            if len(out) not in (2, 3):
                raise ValueError("out must be (k, v) or (k, v, row_start)")
            if len(out) == 3:
                kv_start = _ints("out's row_start", out[2], (b + 1,), device)
            for t in out[:2]:
                if t.dtype is not _BF16 or t.shape != (n_rows, h, D) or t.device != device or not t.is_contiguous():
                    raise ValueError(f"out must be two contiguous bfloat16 [{n_rows}, {h}, {D}] on {device}")
        if kv_start is None:
            kv_start = torch.empty(b + 1, dtype=_INT32, device=device)
        lib = B._lib or B.load()
        st = (lib.oasis_read_kv_q8 if self.bits == 8 else lib.oasis_read_kv_q4)(
            self._shape, self.kv.data_ptr() + layer * self._kv_bytes, self.scale.data_ptr() + layer * self._scale_bytes,
            self.table.data_ptr(), ctx_len.data_ptr(), k_at, ks, v_at, vs, start_at, n_new, only_new, kv_start.data_ptr(),
            out[0].data_ptr(), out[1].data_ptr(), n_rows, self.err.data_ptr(), _current_stream(self._index))
        if st:
            B._check(f"oasis_read_kv_q{self.bits}", st)
        return Rows(out[0], out[1], kv_start)

    def resume(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: Plan, n_held: int, layer: int = 0,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Causal attention of a plan's rows over what their requests hold (lens, before the plan's commit) and
        over each other: q [rows, Hq, 128], k and v [rows, Hkv, 128] in bf16.  n_held: at least the tokens
        that the requests with new rows hold in all, which sizes the scratch and nothing else (a request that does not fit is
        reported to :meth:`check`; its rows and those of requests behind it stay as they are).  Rows of no
        request stay as they are in out (zero where out is allocated here).  The held tokens are read back from
        the pages (:meth:`read`), the new ones are taken as given: call it before :meth:`store`, which in 8
        bits may round a page's earlier tokens again, and before :meth:`commit`."""
        if _current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.resume(q, k, v, plan, n_held, layer, scale, out)
        if q.dim() != 3:
            raise ValueError("q, k and v must be [rows, heads, 128]")
        n, b, hq, hkv, device = q.shape[0], self.batch, self.n_q_heads, self.n_kv_heads, self.device
        qs, ks, vs = _rows("q", q, hq, n, device), _rows("k", k, hkv, n, device), _rows("v", v, hkv, n, device)
        row_start = _ints("plan.row_start", plan.row_start, (b + 1,), device).data_ptr()
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer {layer} of {self.layers}")
        if n_held < 0:
            raise ValueError("n_held must be >= 0")
        if out is None:
            out = torch.zeros((n, hq, D), dtype=_BF16, device=device)
        out_stride = _rows("out", out, hq, n, device)
        if n == 0:
            return out
        ws_bytes = self._resume_bytes + (n + n_held) * hkv * D * 4
        stream = _current_stream(self._index)
        keep = ws_bytes <= _KEPT and not torch._C._cuda_isCurrentStreamCapturing()
        ws = self._resume_scratch.get(stream) if keep else None
        if ws is None or ws.shape[0] < ws_bytes:
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
            if keep:
                self._resume_scratch[stream] = ws
        lib = B._lib or B.load()
        st = (lib.oasis_resume_kv_q8 if self.bits == 8 else lib.oasis_resume_kv_q4)(
            self._shape, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, row_start, n,
            self.kv.data_ptr() + layer * self._kv_bytes, self.scale.data_ptr() + layer * self._scale_bytes,
            self.table.data_ptr(), self.lens.data_ptr(), n_held, _SCALE if scale is None else scale, ws.data_ptr(), ws_bytes,
            out.data_ptr(), out_stride, self.err.data_ptr(), stream)
        if st:
            B._check(f"oasis_resume_kv_q{self.bits}", st)
        return out

    def check(self) -> None:
        """Waits for the device (every stream) and raises if a kernel reported an error; clears the word."""
        torch.cuda.synchronize(self.device)
        bits = int(self.err.item())
        if bits:
            self.err.zero_()
            torch.cuda.synchronize(self.device)  # a call that follows on another stream finds it clear
            names = [n for n in ("BAD_BLOCK", "BAD_SLOT", "NO_SLOT", "BAD_COUNT", "TIMEOUT")
                     if bits & getattr(B, "EW_" + n)]
            raise B.OasisError("paged cache", 1, "device error word: " + ", ".join(names))
