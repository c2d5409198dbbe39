"""The paged cache and beam search of ``libck.so`` (include/ck.h, "a cache in pages" and "beam
search").  As the rest of the binding this module only marshals arguments; what the C side
cannot see (a tensor's type, shape, strides and device) is checked here, and a wrong one raises
ValueError.  Every call returns the library's error number first and enqueues its work on
`stream` (the current one by default) without synchronising.  Arrays of u32 are int32 tensors;
CK_NO_PAGE is -1 in them."""
from __future__ import annotations

import ctypes
from typing import NamedTuple

NO_PAGE = -1
# phase bytes of a batch's status words besides the cache stores' 6, 7 and 8
BAD_SEQUENCE, BAD_PAGE = 1, 2

_vp, _sz, _u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32


class _Cache(ctypes.Structure):
    _fields_ = [("dev_k", _vp), ("dev_v", _vp)] + [(n, _u32) for n in
                                                   ("pages", "layers", "kv_heads", "page", "head_dim")]


class _Batch(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dev_start", "dev_len", "dev_table", "dev_status")] + [
        (n, _u32) for n in ("seqs", "rows", "stride", "max_new", "max_len")]


_cache_p, _batch_p, _size_p = ctypes.POINTER(_Cache), ctypes.POINTER(_Batch), ctypes.POINTER(_sz)

SIGNATURES = {
    "ck_paged_store": ([_cache_p, _u32, _batch_p, _vp, _sz, _vp, _sz, _vp, _sz, _u32, _vp, _u32, _u32,
                        ctypes.c_int, _vp, _vp], ctypes.c_int),
    "ck_paged_attention_work": ([_cache_p, _batch_p, _u32, _size_p], ctypes.c_int),
    "ck_paged_attention": ([_cache_p, _u32, _batch_p, _vp, _sz, _u32, _vp, _u32, _vp, _vp, _sz, _vp],
                           ctypes.c_int),
    "ck_pages_work": ([_cache_p, _u32, _u32, _size_p], ctypes.c_int),
    "ck_pages_fork": ([_cache_p, _u32, _vp, _vp, _u32, _vp, _vp, _u32, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
                      ctypes.c_int),
    "ck_pages_compact": ([_cache_p, _u32, _vp, _vp, _u32, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "ck_beam_work": ([_u32, _u32, _u32, _size_p], ctypes.c_int),
    "ck_beam_select": ([_vp, _sz, _u32, _u32, _u32, _vp, _vp, _vp, _u32, _u32, _vp, _vp, _vp, _vp, _vp, _sz,
                        _vp], ctypes.c_int),
    "ck_host_log_sum": ([ctypes.c_uint64], ctypes.c_int64),
}


def _lib():
    from . import lib
    return lib()


def _torch():
    import torch
    return torch


def _check(name, t, dtype, shape, device):
    """A contiguous tensor of the type and shape (None: any extent) on the device."""
    if t.dtype is not dtype or t.dim() != len(shape) or not t.is_contiguous() or any(
            w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name}: want a contiguous {dtype} tensor of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    _check_device(name, t, device)


def _check_device(name, t, device):
    if t.device.type != "cuda" or t.device.index != device:
        raise ValueError(f"{name}: not on CUDA device {device} ({t.device})")


def _check_rows(name, t, rows, device):
    """int64 rows whose elements follow one another (the rows themselves may be further apart)."""
    torch = _torch()
    if t.dtype is not torch.int64 or t.dim() != 2 or t.shape[0] != rows or (t.shape[1] > 1 and t.stride(1) != 1) or (
            rows > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name}: want {rows} int64 rows of contiguous elements, got {t.dtype} {tuple(t.shape)} "
                         f"strides {t.stride()}")
    _check_device(name, t, device)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] + (t.shape[1] & 1)


def _new(stream, *args, **kw):
    """A tensor from the allocator's pool of the stream the call runs on."""
    torch = _torch()
    if stream is None:
        return torch.empty(*args, **kw)
    with torch.cuda.stream(stream):
        return torch.empty(*args, **kw)


def _raw(stream):
    torch = _torch()
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


class PagedCache:
    """Key and value pools: int32 [pages][layers][kv heads][page][head], on one device."""

    def __init__(self, k, v):
        torch = _torch()
        _check("k", k, torch.int32, (None,) * 5, k.device.index)
        _check("v", v, torch.int32, k.shape, k.device.index)
        self.k, self.v, self.device = k, v, k.device.index
        self.pages, self.layers, self.kv_heads, self.page, self.head_dim = k.shape
        self._c = _Cache(k.data_ptr(), v.data_ptr(), *k.shape)

    @classmethod
    def empty(cls, pages, layers, kv_heads, page, head_dim):
        """Pools of zeros on the current device."""
        torch = _torch()
        shape = (pages, layers, kv_heads, page, head_dim)
        return cls(*(torch.zeros(shape, dtype=torch.int32, device="cuda") for _ in range(2)))


class PagedBatch:
    """New tokens of several sequences (ck_paged_batch): table int32 [seqs][stride], lens int32
    [seqs], starts int32 [seqs + 1], status int64 [seqs] (None: a new one, set to -1).  The tensors
    are read by the kernels, so they may be refilled between calls; max_new and max_len bound what
    they may say."""

    def __init__(self, table, lens, starts, status, rows, max_new, max_len):
        torch = _torch()
        self.device = table.device.index
        _check("table", table, torch.int32, (None, None), self.device)
        seqs = table.shape[0]
        _check("lens", lens, torch.int32, (seqs,), self.device)
        _check("starts", starts, torch.int32, (seqs + 1,), self.device)
        if status is None:
            status = torch.full((seqs,), -1, dtype=torch.int64, device=table.device)
        _check("status", status, torch.int64, (seqs,), self.device)
        self.table, self.lens, self.starts, self.status, self.rows = table, lens, starts, status, rows
        self._c = _Batch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), status.data_ptr(), seqs, rows,
                         table.shape[1], max_new, max_len)

    def errors(self):
        """The status words on the host as (position, layer, phase, element), None where there is
        none (synchronises)."""
        return [None if w == -1 else ((w >> 44) & 0xFFFFF, (w >> 32) & 0xFFF, (w >> 24) & 0xFF, w & 0xFFFFFF)
                for w in self.status.tolist()]


def _devices(cache, batch):
    device = _torch().cuda.current_device()
    if cache.device != device or batch.device != device:
        raise ValueError("the cache and the batch are not both on the current CUDA device")
    return device


def _out(out, rows, cols, device, stream, like):
    torch = _torch()
    if out is None:
        return _new(stream, (rows, cols), dtype=torch.int64, device=like.device)
    _check("out", out, torch.int64, (rows, cols), device)
    return out


def paged_store(cache, layer, batch, q, k, v, rope, half=False, out=None, stream=None):
    """Rotary and the checked stores of a batch's new rows (ck_paged_store).  q, k, v: int64 rows,
    which may be column ranges of one tensor; rope: int32 [positions][rot / 2][2].  Returns (rc,
    rotated queries)."""
    torch = _torch()
    device = _devices(cache, batch)
    hd = cache.head_dim
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_rows(name, t, batch.rows, device)
    _check("rope", rope, torch.int32, (None, None, 2), device)
    if q.shape[1] % hd or k.shape[1] != cache.kv_heads * hd or v.shape[1] != k.shape[1]:
        raise ValueError("q, k and v: columns do not match the cache's heads")
    out = _out(out, batch.rows, q.shape[1], device, stream, q)
    rc = _lib().ck_paged_store(cache._c, layer, batch._c, q.data_ptr(), _row_stride(q), k.data_ptr(),
                               _row_stride(k), v.data_ptr(), _row_stride(v), q.shape[1] // hd, rope.data_ptr(),
                               rope.shape[0], 2 * rope.shape[1], int(half), out.data_ptr(), _raw(stream))
    return rc, out


def paged_attention_work(cache, batch, heads):
    """Scratch for paged_attention on the current stream, as large as the batch's bounds need."""
    torch = _torch()
    n = _sz()
    rc = _lib().ck_paged_attention_work(cache._c, batch._c, heads, ctypes.byref(n))
    if rc:
        from . import CkError
        raise CkError(rc, "ck_paged_attention_work")
    return torch.empty(n.value, dtype=torch.uint8, device=cache.k.device)


def paged_attention(cache, layer, batch, q, exp_table, inv_sqrt, out=None, work=None, stream=None):
    """Attention of a batch's new rows over their sequences' pages (ck_paged_attention).  q: int64
    rows of rotated queries; exp_table: int32 [4097].  Returns (rc, outputs)."""
    torch = _torch()
    device = _devices(cache, batch)
    hd = cache.head_dim
    _check_rows("q", q, batch.rows, device)
    _check("exp_table", exp_table, torch.int32, (4097,), device)
    if q.shape[1] == 0 or q.shape[1] % (hd * cache.kv_heads):
        raise ValueError("q: columns are no multiple of the cache's heads")
    heads = q.shape[1] // hd
    out = _out(out, batch.rows, q.shape[1], device, stream, q)
    if work is None:
        if stream is None:
            work = paged_attention_work(cache, batch, heads)
        else:
            with torch.cuda.stream(stream):
                work = paged_attention_work(cache, batch, heads)
    _check("work", work, torch.uint8, (None,), device)
    rc = _lib().ck_paged_attention(cache._c, layer, batch._c, q.data_ptr(), _row_stride(q), heads,
                                   exp_table.data_ptr(), inv_sqrt, out.data_ptr(), work.data_ptr(), work.numel(),
                                   _raw(stream))
    return rc, out


class Fork(NamedTuple):
    table: object   # int32 [rows][stride]
    lens: object    # int32 [rows], grown
    status: object  # int32 [rows]


class Compact(NamedTuple):
    table: object
    used: object    # int32 scalar
    status: object


class PagePlan:
    """Scratch for moving the pages of up to `rows` sequences with tables of `stride` entries.
    Calls on one plan must follow one another on one stream (or be ordered by the caller)."""

    def __init__(self, cache, rows, stride):
        torch = _torch()
        n = _sz()
        rc = _lib().ck_pages_work(cache._c, rows, stride, ctypes.byref(n))
        if rc:
            from . import CkError
            raise CkError(rc, "ck_pages_work")
        self.cache, self.rows, self.stride = cache, rows, stride
        self._work = torch.empty(n.value, dtype=torch.uint8, device=cache.k.device)

    def _begin(self, lens, table):
        torch = _torch()
        device = torch.cuda.current_device()
        _check_device("cache", self.cache.k, device)
        _check("table", table, torch.int32, (None, self.stride), device)
        _check("lens", lens, torch.int32, (table.shape[0],), device)
        return device

    def fork(self, parent, lens, table, grow, held=None, stream=None):
        """ck_pages_fork: output row r takes over input row parent[r] (-1: none) and gets pages for
        grow[r] more positions; held (uint8 [pages]) marks pages of others.  Returns (rc, Fork)."""
        torch = _torch()
        device = self._begin(lens, table)
        _check("parent", parent, torch.int32, (None,), device)
        rows = parent.shape[0]
        if rows > self.rows:
            raise ValueError(f"parent: {rows} rows, the plan has room for {self.rows}")
        _check("grow", grow, torch.int32, (rows,), device)
        if held is not None:
            _check("held", held, torch.uint8, (self.cache.pages,), device)
        flat = _new(stream, rows * (self.stride + 2), dtype=torch.int32, device=table.device)
        out, new_lens, status = flat.split((rows * self.stride, rows, rows))
        rc = _lib().ck_pages_fork(self.cache._c, table.shape[0], lens.data_ptr(), table.data_ptr(), rows,
                                  parent.data_ptr(), grow.data_ptr(), self.stride,
                                  None if held is None else held.data_ptr(), new_lens.data_ptr(), out.data_ptr(),
                                  status.data_ptr(), self._work.data_ptr(), self._work.numel(), _raw(stream))
        return rc, Fork(out.view(rows, self.stride), new_lens, status)

    def compact(self, lens, table, stream=None):
        """ck_pages_compact: the rows' pages move to the lowest page numbers.  Returns (rc, Compact)."""
        torch = _torch()
        self._begin(lens, table)
        rows = table.shape[0]
        if rows > self.rows:
            raise ValueError(f"table: {rows} rows, the plan has room for {self.rows}")
        flat = _new(stream, rows * (self.stride + 1) + 1, dtype=torch.int32, device=table.device)
        out, status, used = flat.split((rows * self.stride, rows, 1))
        rc = _lib().ck_pages_compact(self.cache._c, rows, lens.data_ptr(), table.data_ptr(), self.stride,
                                     out.data_ptr(), used.data_ptr(), status.data_ptr(), self._work.data_ptr(),
                                     self._work.numel(), _raw(stream))
        return rc, Compact(out.view(rows, self.stride), used[0], status)


class Beams(NamedTuple):
    scores: object  # int64 [groups * beams]
    parent: object  # int32: the row extended, -1 for none
    token: object   # int32
    done: object    # uint8


class BeamPlan:
    """Scratch for the selection of `groups` searches of `beams` beams.  Calls on one plan must
    follow one another on one stream (or be ordered by the caller)."""

    def __init__(self, groups, beams, vocab):
        torch = _torch()
        n = _sz()
        rc = _lib().ck_beam_work(groups, beams, vocab, ctypes.byref(n))
        if rc:
            from . import CkError
            raise CkError(rc, "ck_beam_work")
        self.groups, self.beams, self.vocab = groups, beams, vocab
        self._work = torch.empty(n.value, dtype=torch.uint8, device="cuda")

    def select(self, logits, scores, done, exp_table, stop_tokens=False, done_token=0, stream=None):
        """ck_beam_select: the next beams of every search from logits int64 [groups * beams][vocab]
        (rows may be further apart), scores int64 and done uint8.  Returns (rc, Beams)."""
        torch = _torch()
        device = torch.cuda.current_device()
        rows = self.groups * self.beams
        _check_device("plan", self._work, device)
        _check_rows("logits", logits, rows, device)
        if logits.shape[1] != self.vocab:
            raise ValueError(f"logits: {logits.shape[1]} columns, the plan is for {self.vocab}")
        _check("scores", scores, torch.int64, (rows,), device)
        _check("done", done, torch.uint8, (rows,), device)
        _check("exp_table", exp_table, torch.int32, (4097,), device)
        flat = _new(stream, rows * 17, dtype=torch.uint8, device=logits.device)
        new_scores, parent, token, new_done = flat.split((8 * rows, 4 * rows, 4 * rows, rows))
        rc = _lib().ck_beam_select(logits.data_ptr(), _row_stride(logits), self.groups, self.beams, self.vocab,
                                   scores.data_ptr(), done.data_ptr(), exp_table.data_ptr(), int(stop_tokens),
                                   done_token, new_scores.data_ptr(), parent.data_ptr(), token.data_ptr(),
                                   new_done.data_ptr(), self._work.data_ptr(), self._work.numel(), _raw(stream))
        return rc, Beams(new_scores.view(torch.int64), parent.view(torch.int32), token.view(torch.int32), new_done)


def host_log_sum(z: int) -> int:
    """Host build of the logarithm of a sum of exponentials as ck_beam_select takes it."""
    return int(_lib().ck_host_log_sum(z))
