"""The paged cache, beam search and sampling of ``libck.so`` (include/ck.h, "a cache in pages", "beam
search" and "sampling").  As the rest of the binding this module only marshals arguments; what the C side
cannot see (a tensor's type, shape, strides and device) is checked here, and a wrong one raises
ValueError.  Every call returns the library's error number first and enqueues its work on
`stream` (the current one by default) without synchronising.  Arrays of u32 are int32 tensors;
CK_NO_PAGE is -1 in them.  A number that is no u32 raises ValueError too."""
from __future__ import annotations

import ctypes
import operator
from typing import NamedTuple

import torch

from . import CkError, lib

NO_PAGE = -1
# phase bytes of a batch's status words besides the cache stores' 6, 7 and 8
BAD_SEQUENCE, BAD_PAGE = 1, 2
# marks of PagePlan.fork's held: not handed out; and of a sequence that lives on outside the call
PAGE_RESERVED, PAGE_SHARED = 1, 2
# Beams.done of a search that failed (a wait of its kernel ran out)
BEAM_FAILED = 255
# a sampled row without a token
NO_TOKEN = -1

_vp, _sz, _u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32
_device = torch.cuda.current_device


class _Cache(ctypes.Structure):
    _fields_ = [("dev_k", _vp), ("dev_v", _vp)] + [(n, _u32) for n in
                                                   ("pages", "layers", "kv_heads", "page", "head_dim")]


class _Batch(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dev_start", "dev_len", "dev_table", "dev_status")] + [
        (n, _u32) for n in ("seqs", "rows", "stride", "max_new", "max_len")]


class _Window(ctypes.Structure):
    _fields_ = [("sinks", _u32), ("window", _u32)]


class Window(NamedTuple):
    """What a row of attention sees: the sequence's first `sinks` positions and its last `window`, its own
    among them."""
    sinks: int
    window: int


def _window(w):
    """A window as the library takes it (None: the whole cache)."""
    if w is None:
        return None
    sinks, window = w
    return ctypes.byref(_Window(_u32_of("sinks", sinks), _u32_of("window", window)))


def _windows(w, layers):
    """A window for every layer (one stands for all of them)."""
    if w is None:
        return None
    each = [w] * layers if isinstance(w, Window) else list(w)
    if len(each) != layers or not all(isinstance(one, tuple) and len(one) == 2 for one in each):
        raise ValueError(f"window: want a Window, or one for each of the model's {layers} layers, got {w!r}")
    return (_Window * layers)(*(_Window(_u32_of("sinks", s), _u32_of("window", n)) for s, n in each))


def _u32_of(name, value):
    """The number as the library takes it (ctypes would cut it to its low 32 bits)."""
    value = operator.index(value)
    if not 0 <= value <= 0xFFFFFFFF:
        raise ValueError(f"{name}: want a number from 0 to 2^32 - 1, got {value}")
    return value


def _check(name, t, dtype, shape, device):
    """A contiguous tensor of the type and shape on the device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name}: want a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {device}, "
                         f"got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _check_rows(name, t, rows, device):
    """int64 rows whose elements follow one another (the rows themselves may be further apart);
    the words from one row to the next."""
    if t.dtype is torch.int64 and t.dim() == 2 and t.get_device() == device:
        n, cols = t.shape
        step, inner = t.stride()
        if n == rows and (inner == 1 or cols <= 1) and (step >= cols or rows == 1):
            return step if rows > 1 else cols + (cols & 1)
    raise ValueError(f"{name}: want {rows} int64 rows of contiguous elements on CUDA device {device}, got {t.dtype} "
                     f"{tuple(t.shape)} strides {t.stride()} on {t.device}")


def _empty(stream, shape, dtype, device):
    """A tensor from the allocator's pool of the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _made_on(stream, make, *args):
    """What make(*args) allocates, from the pool of the stream the call runs on."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _keep(stream, *tensors):
    """The tensors stay in use on the stream, whatever becomes of them after the call."""
    if stream is not None:
        for t in tensors:
            t.record_stream(stream)


def _raw(device):
    return torch._C._cuda_getCurrentRawStream(device)


def _allocated(*tensors):
    """What an object allocated itself: the stream it did so on (None: not on a GPU), and the tensors."""
    return _raw(tensors[0].get_device()) if tensors[0].is_cuda else None, tensors


def _on(stream, device, *owners):
    """The stream a call runs on, as the library takes it.  What the owners allocated themselves stays
    in use there, as on a `stream` given (_keep): their caller has no tensor to record."""
    if stream is not None:
        return stream.cuda_stream
    raw = _raw(device)
    for o in owners:
        if o._home is not None and o._home != raw:
            for t in o._made:
                t.record_stream(torch.cuda.current_stream(device))
    return raw


def _size(name, *args):
    n = _sz()
    rc = getattr(lib(), name)(*args, ctypes.byref(n))
    if rc:
        raise CkError(rc, name)
    return n.value


class PagedCache:
    """Key and value pools: int32 [pages][layers][kv heads][page][head], on one device."""

    def __init__(self, k, v):
        if k.dim() != 5 or not k.is_cuda:
            raise ValueError(f"k: want a five-dimensional CUDA tensor, got {tuple(k.shape)} on {k.device}")
        self.device = k.get_device()
        _check("k", k, torch.int32, k.shape, self.device)
        _check("v", v, torch.int32, k.shape, self.device)
        self.k, self.v = k, v
        self.pages, self.layers, self.kv_heads, self.page, self.head_dim = k.shape
        self._struct = _Cache(k.data_ptr(), v.data_ptr(), *k.shape)
        self._c = ctypes.addressof(self._struct)
        self._tensors = k, v
        self._home, self._made = None, ()  # (the caller's own)

    @classmethod
    def empty(cls, pages, layers, kv_heads, page, head_dim):
        """Pools of zeros on the current device."""
        shape = (pages, layers, kv_heads, page, head_dim)
        cache = cls(*(torch.zeros(shape, dtype=torch.int32, device="cuda") for _ in range(2)))
        cache._home, cache._made = _allocated(*cache._tensors)
        return cache


class PagedBatch:
    """New tokens of several sequences (ck_paged_batch): table int32 [seqs][stride], lens int32
    [seqs], starts int32 [seqs + 1], status int64 [seqs] (None: a new one, set to -1).  The tensors
    are read by the kernels, so they may be refilled between calls; max_new and max_len bound what
    they may say."""

    def __init__(self, table, lens, starts, status, rows, max_new, max_len):
        if table.dim() != 2 or not table.is_cuda:
            raise ValueError(f"table: want a two-dimensional CUDA tensor, got {tuple(table.shape)} on {table.device}")
        self.device = table.get_device()
        _check("table", table, torch.int32, table.shape, self.device)
        seqs = table.shape[0]
        _check("lens", lens, torch.int32, (seqs,), self.device)
        _check("starts", starts, torch.int32, (seqs + 1,), self.device)
        self._home, self._made = None, ()
        if status is None:
            status = torch.full((seqs,), -1, dtype=torch.int64, device=table.device)
            self._home, self._made = _allocated(status)
        _check("status", status, torch.int64, (seqs,), self.device)
        rows, max_new, max_len = _u32_of("rows", rows), _u32_of("max_new", max_new), _u32_of("max_len", max_len)
        self.table, self.lens, self.starts, self.status, self.rows = table, lens, starts, status, rows
        self._struct = _Batch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), status.data_ptr(), seqs, rows,
                              table.shape[1], max_new, max_len)
        self._c = ctypes.addressof(self._struct)
        self._tensors = table, lens, starts, status

    def errors(self):
        """The status words on the host as (position, layer, phase, element), None where there is
        none (synchronises)."""
        return [None if w == -1 else ((w >> 44) & 0xFFFFF, (w >> 32) & 0xFFF, (w >> 24) & 0xFF, w & 0xFFFFFF)
                for w in self.status.tolist()]


def _call_device(stream):
    """The current device, which a stream given has to be on as well."""
    device = _device()
    if stream is not None and stream.device.index != device:
        raise ValueError(f"stream: want one on the current CUDA device {device}, got {stream.device}")
    return device


def _devices(cache, batch, stream):
    device = _call_device(stream)
    if cache.device != device or batch.device != device:
        raise ValueError("the cache and the batch are not both on the current CUDA device")
    return device


def paged_store(cache, layer, batch, q, k, v, rope, half=False, out=None, stream=None):
    """Rotary and the checked stores of a batch's new rows (ck_paged_store).  q, k, v: int64 rows,
    which may be column ranges of one tensor; rope: int32 [positions][rot / 2][2].  Returns (rc,
    rotated queries)."""
    device, rows, hd = _devices(cache, batch, stream), batch.rows, cache.head_dim
    q_step = _check_rows("q", q, rows, device)
    k_step = _check_rows("k", k, rows, device)
    v_step = _check_rows("v", v, rows, device)
    if rope.dim() != 3 or rope.shape[2] != 2:
        raise ValueError(f"rope: want [positions][rot / 2][2], got {tuple(rope.shape)}")
    _check("rope", rope, torch.int32, rope.shape, device)
    cols, kv_cols = q.shape[1], cache.kv_heads * hd
    if not hd or cols % hd or k.shape[1] != kv_cols or v.shape[1] != kv_cols:
        raise ValueError("q, k and v: columns do not match the cache's heads")
    if out is None:
        out = _empty(stream, (rows, cols), torch.int64, device)
    else:
        _check("out", out, torch.int64, (rows, cols), device)
    _keep(stream, q, k, v, rope, out, *cache._tensors, *batch._tensors)
    rc = lib().ck_paged_store(cache._c, _u32_of("layer", layer), batch._c, q.data_ptr(), q_step, k.data_ptr(), k_step, v.data_ptr(),
                              v_step, cols // hd, rope.data_ptr(), rope.shape[0], 2 * rope.shape[1], half,
                              out.data_ptr(), _on(stream, device, cache, batch))
    return rc, out


def paged_attention_work(cache, batch, heads, stream=None, window=None):
    """Scratch for paged_attention on the stream, as large as the batch's bounds and the window need."""
    device = _devices(cache, batch, stream)
    return _empty(stream, _size("ck_paged_window_attention_work", cache._c, batch._c, heads, _window(window)), torch.uint8,
                  device)


def paged_attention(cache, layer, batch, q, exp_table, inv_sqrt, out=None, work=None, stream=None, window=None):
    """Attention of a batch's new rows over their sequences' pages (ck_paged_attention), or over a
    Window of them (ck_paged_window_attention).  q: int64 rows of rotated queries; exp_table: int32
    [4097].  Returns (rc, outputs)."""
    device, rows, hd = _devices(cache, batch, stream), batch.rows, cache.head_dim
    step = _check_rows("q", q, rows, device)
    _check("exp_table", exp_table, torch.int32, (4097,), device)
    cols = q.shape[1]
    if cols == 0 or hd * cache.kv_heads == 0 or cols % (hd * cache.kv_heads):
        raise ValueError("q: columns are no multiple of the cache's heads")
    if out is None:
        out = _empty(stream, (rows, cols), torch.int64, device)
    else:
        _check("out", out, torch.int64, (rows, cols), device)
    if work is None:
        work = paged_attention_work(cache, batch, cols // hd, stream, window)
    else:
        _check("work", work, torch.uint8, (work.numel(),), device)
    _keep(stream, q, exp_table, out, work, *cache._tensors, *batch._tensors)
    rc = lib().ck_paged_window_attention(cache._c, _u32_of("layer", layer), batch._c, q.data_ptr(), step, cols // hd,
                                         _window(window), exp_table.data_ptr(), _u32_of("inv_sqrt", inv_sqrt),
                                         out.data_ptr(), work.data_ptr(), work.numel(), _on(stream, device, cache, batch))
    return rc, out


def turn_paged_work(model, cache, batch, stream=None, window=None):
    device = _devices(cache, batch, stream)
    each = _windows(window, model.config["layers"])
    return _empty(stream, _size("ck_turn_paged_window_work", model._h, cache._c, batch._c, each), torch.uint8, device)


def turn_paged(model, cache, batch, tokens, logits=None, work=None, stream=None, window=None):
    device, seqs, vocab = _devices(cache, batch, stream), batch.lens.shape[0], model.config["vocab"]
    if model.mem.get_device() != device:
        raise ValueError("the model is not on the current CUDA device")
    _check("tokens", tokens, torch.int32, (batch.rows,), device)
    if logits is None:
        logits = _empty(stream, (seqs, vocab), torch.int64, device)
    step = _check_rows("logits", logits, seqs, device)
    if logits.shape[1] != vocab:
        raise ValueError(f"logits: {logits.shape[1]} columns, the vocabulary is {vocab}")
    if window is not None and not isinstance(window, Window):
        window = list(window)
    each = _windows(window, model.config["layers"])
    if work is None:
        work = turn_paged_work(model, cache, batch, stream, window)
    else:
        _check("work", work, torch.uint8, (work.numel(),), device)
    _keep(stream, model.mem, tokens, logits, work, *cache._tensors, *batch._tensors)
    rc = lib().ck_turn_paged_window(model._h, cache._c, batch._c, each, tokens.data_ptr(), logits.data_ptr(), step,
                                    work.data_ptr(), work.numel(), _on(stream, device, model, cache, batch))
    return rc, logits


class Fork(NamedTuple):
    table: object   # int32 [rows][stride]
    lens: object    # int32 [rows], grown
    status: object  # int32 [rows]


class Advance(NamedTuple):
    table: object      # int32 [seqs][stride]
    lens: object       # int32 [seqs], grown
    starts: object     # int32 [seqs + 1]
    slots: object      # int64 [rows], -1 for none
    positions: object  # int32 [rows], -1 for none
    status: object     # int32 [seqs]


def _advance_outputs(table, lens, rows):
    return (torch.empty_like(table), torch.empty_like(lens), lens.new_empty(lens.shape[0] + 1),
            lens.new_empty(rows, dtype=torch.int64), lens.new_empty(rows), torch.empty_like(lens))


class Compact(NamedTuple):
    table: object
    used: object    # int32 scalar
    status: object


class PagePlan:
    """Scratch for moving the pages of up to `rows` sequences with tables of `stride` entries.
    Calls on one plan must follow one another on one stream (or be ordered by the caller)."""

    def __init__(self, cache, rows, stride):
        self.cache, self.rows, self.stride = cache, _u32_of("rows", rows), _u32_of("stride", stride)
        self._work = torch.empty(_size("ck_pages_work", cache._c, rows, stride), dtype=torch.uint8,
                                 device=cache.k.device)
        self._args = self._work.data_ptr(), self._work.numel()
        self._home, self._made = _allocated(self._work)

    def _begin(self, lens, table, stream):
        device, rows = _call_device(stream), table.shape[0]
        if self.cache.device != device:
            raise ValueError("the cache is not on the current CUDA device")
        _check("table", table, torch.int32, (rows, self.stride), device)
        _check("lens", lens, torch.int32, (rows,), device)
        return device, rows

    def fork(self, parent, lens, table, grow, held=None, stream=None, window=None):
        """ck_pages_fork: output row r takes over input row parent[r] (-1: none) and gets pages for
        grow[r] more positions; held (uint8 [pages]): PAGE_RESERVED pages are not handed out,
        PAGE_SHARED ones, of sequences that live on outside the call, are also copied where a row
        has them part-filled.  window: the Window of sequences that advance() moves on
        (ck_pages_window_fork).  Returns (rc, Fork)."""
        device, rows_in = self._begin(lens, table, stream)
        rows = parent.numel()
        if rows > self.rows:
            raise ValueError(f"parent: {rows} rows, the plan has room for {self.rows}")
        _check("parent", parent, torch.int32, (rows,), device)
        _check("grow", grow, torch.int32, (rows,), device)
        if held is not None:
            _check("held", held, torch.uint8, (self.cache.pages,), device)
        view = _window(window)
        _keep(stream, self._work, parent, lens, table, grow, *(() if held is None else (held,)), *self.cache._tensors)
        out = _empty(stream, (rows, self.stride), torch.int32, device)
        new_lens, status = _empty(stream, (rows,), torch.int32, device), _empty(stream, (rows,), torch.int32, device)
        rc = lib().ck_pages_window_fork(self.cache._c, rows_in, lens.data_ptr(), table.data_ptr(), rows,
                                        parent.data_ptr(), grow.data_ptr(), self.stride, view,
                                        None if held is None else held.data_ptr(), new_lens.data_ptr(), out.data_ptr(),
                                        status.data_ptr(), *self._args, _on(stream, device, self, self.cache))
        return rc, Fork(out, new_lens, status)

    def advance(self, lens, table, new, rows, window=None, held=None, stream=None):
        """ck_pages_advance: every sequence gives back the pages behind its Window (None: it keeps all) and
        gets pages for new[s] more positions, at most `rows` of them together; held (uint8 [pages]):
        nonzero pages are not handed out.  A sequence whose part-filled page another entry names, or that
        is PAGE_SHARED, gets no rows (status 10).  The outputs' tensors are a PagedBatch's.  Returns (rc,
        Advance)."""
        device, seqs = self._begin(lens, table, stream)
        if seqs > self.rows:
            raise ValueError(f"table: {seqs} rows, the plan has room for {self.rows}")
        _check("new", new, torch.int32, (seqs,), device)
        if held is not None:
            _check("held", held, torch.uint8, (self.cache.pages,), device)
        rows = _u32_of("rows", rows)
        if not 1 <= rows <= 2**20:
            raise ValueError(f"rows: want a number from 1 to 2^20, got {rows}")
        view = _window(window)
        if stream is not None:
            _keep(stream, self._work, lens, table, new, *(() if held is None else (held,)), *self.cache._tensors)
        got = out, new_lens, starts, slots, positions, status = _made_on(stream, _advance_outputs, table, lens, rows)
        rc = lib().ck_pages_advance(self.cache._c, seqs, lens.data_ptr(), table.data_ptr(), new.data_ptr(), self.stride,
                                    view, None if held is None else held.data_ptr(), rows, new_lens.data_ptr(),
                                    out.data_ptr(), starts.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                                    status.data_ptr(), *self._args, _on(stream, device, self, self.cache))
        return rc, Advance(*got)

    def compact(self, lens, table, stream=None, window=None):
        """ck_pages_compact: the rows' pages move to the lowest page numbers; window: as fork's
        (ck_pages_window_compact).  Returns (rc, Compact)."""
        device, rows = self._begin(lens, table, stream)
        if rows > self.rows:
            raise ValueError(f"table: {rows} rows, the plan has room for {self.rows}")
        view = _window(window)
        _keep(stream, self._work, lens, table, *self.cache._tensors)
        out = _empty(stream, (rows, self.stride), torch.int32, device)
        status = _empty(stream, (rows,), torch.int32, device)
        used = _empty(stream, (), torch.int32, device)
        rc = lib().ck_pages_window_compact(self.cache._c, rows, lens.data_ptr(), table.data_ptr(), self.stride, view,
                                           out.data_ptr(), used.data_ptr(), status.data_ptr(), *self._args,
                                           _on(stream, device, self, self.cache))
        return rc, Compact(out, used, status)


class Beams(NamedTuple):
    scores: object  # int64 [groups * beams]
    parent: object  # int32: the row extended, -1 for none
    token: object   # int32
    done: object    # uint8: 1 ended, BEAM_FAILED everywhere in a search that failed


class BeamPlan:
    """Scratch for the selection of `groups` searches of `beams` beams.  Calls on one plan must
    follow one another on one stream (or be ordered by the caller)."""

    def __init__(self, groups, beams, vocab):
        self.groups, self.beams = _u32_of("groups", groups), _u32_of("beams", beams)
        self.vocab = _u32_of("vocab", vocab)
        self._work = torch.empty(_size("ck_beam_work", groups, beams, vocab), dtype=torch.uint8, device="cuda")
        self._args = self._work.data_ptr(), self._work.numel()
        self._device = self._work.get_device()
        self._home, self._made = _allocated(self._work)

    def select(self, logits, scores, done, exp_table, stop_tokens=False, done_token=0, stream=None):
        """ck_beam_select: the next beams of every search from logits int64 [groups * beams][vocab]
        (rows may be further apart), scores int64 and done uint8.  Returns (rc, Beams)."""
        device, rows = _call_device(stream), self.groups * self.beams
        if self._device != device:
            raise ValueError("the plan is not on the current CUDA device")
        step = _check_rows("logits", logits, rows, device)
        if logits.shape[1] != self.vocab:
            raise ValueError(f"logits: {logits.shape[1]} columns, the plan is for {self.vocab}")
        _check("scores", scores, torch.int64, (rows,), device)
        _check("done", done, torch.uint8, (rows,), device)
        _check("exp_table", exp_table, torch.int32, (4097,), device)
        _keep(stream, self._work, logits, scores, done, exp_table)
        new_scores = _empty(stream, (rows,), torch.int64, device)
        parent, token = _empty(stream, (rows,), torch.int32, device), _empty(stream, (rows,), torch.int32, device)
        new_done = _empty(stream, (rows,), torch.uint8, device)
        rc = lib().ck_beam_select(logits.data_ptr(), step, self.groups, self.beams, self.vocab, scores.data_ptr(),
                                  done.data_ptr(), exp_table.data_ptr(), stop_tokens,
                                  _u32_of("done_token", done_token),
                                  new_scores.data_ptr(), parent.data_ptr(), token.data_ptr(), new_done.data_ptr(),
                                  *self._args, _on(stream, device, self))
        return rc, Beams(new_scores, parent, token, new_done)


class Samples(NamedTuple):
    token: object  # int32 [rows], NO_TOKEN for none
    prob: object   # int32 [rows], 24 fraction bits
    kept: object   # int32 [rows]


def _three(t):
    return torch.empty_like(t), torch.empty_like(t), torch.empty_like(t)


def sample(logits, temperature, random, exp_table, top_k=None, top_p=None, min_p=None, stream=None):
    """A token of every row (ck_sample): logits int64 [rows][vocab] (rows may be further apart),
    temperature int32 [rows] (16 fraction bits), random int64 [rows] (all 64 bits count), exp_table
    int32 [4097]; top_k, top_p and min_p int32 [rows] (the latter two with 24 fraction bits) or None.
    Returns (rc, Samples)."""
    device = _call_device(stream)
    if logits.dim() != 2:
        raise ValueError(f"logits: want two dimensions, got {tuple(logits.shape)}")
    rows, vocab = logits.shape
    step, each = _check_rows("logits", logits, rows, device), (rows,)
    _check("temperature", temperature, torch.int32, each, device)
    _check("random", random, torch.int64, each, device)
    _check("exp_table", exp_table, torch.int32, (4097,), device)
    k = p = m = None
    if top_k is not None:
        _check("top_k", top_k, torch.int32, each, device)
        k = top_k.data_ptr()
    if top_p is not None:
        _check("top_p", top_p, torch.int32, each, device)
        p = top_p.data_ptr()
    if min_p is not None:
        _check("min_p", min_p, torch.int32, each, device)
        m = min_p.data_ptr()
    if stream is not None:
        _keep(stream, logits, temperature, random, exp_table, *(f for f in (top_k, top_p, min_p) if f is not None))
    token, prob, kept = _made_on(stream, _three, temperature)
    rc = lib().ck_sample(logits.data_ptr(), step, rows, vocab, temperature.data_ptr(), k, p, m, random.data_ptr(),
                         exp_table.data_ptr(), token.data_ptr(), prob.data_ptr(), kept.data_ptr(), _on(stream, device))
    return rc, Samples(token, prob, kept)


def set_beam_wait_limit(polls: int) -> int:
    """The process's limit on a row's wait for its cluster's maxima (ck_set_beam_wait_limit)."""
    return lib().ck_set_beam_wait_limit(_u32_of("polls", polls))


def host_sample_place(distance: int, temperature: int) -> int:
    """Host build of a distance's place in the exponential table as ck_sample takes it."""
    return int(lib().ck_host_sample_place(_u32_of("distance", distance), _u32_of("temperature", temperature)))


def host_log_sum(z: int) -> int:
    """Host build of the logarithm of a sum of exponentials as ck_beam_select takes it."""
    return int(lib().ck_host_log_sum(z))
