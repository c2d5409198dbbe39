"""What windowed attention, the page tables' step between passes and sampling refuse, and their host
routines: no GPU needed (every refusal is decided from the arguments alone, before any device
call)."""
import ctypes

import numpy as np
import pytest

from test_paged import ADDR, BAD_BATCHES, BAD_CACHES, attention_args, batch, cache, call, ck, compact_args, fork_args  # noqa: F401


def window(ck, sinks=4, size=16):
    return ck.paged._Window(sinks, size)


def window_args(ck):
    args = attention_args(ck)
    out = {}
    for name, value in args.items():
        if name == "exp":
            out["window"] = window(ck)
        out[name] = value
    return out


@pytest.mark.parametrize("bad", BAD_CACHES + BAD_BATCHES, ids=str)
def test_wrong_caches_and_batches_are_refused(ck, bad):
    key = "cache" if bad.keys() & {n for n, _ in ck.paged._Cache._fields_} else "batch"
    value = cache(ck, **bad) if key == "cache" else batch(ck, **bad)
    assert call(ck, "ck_paged_window_attention", window_args(ck), **{key: value}) == 10


@pytest.mark.parametrize("bad", [dict(cache=None), dict(layer=2), dict(batch=None), dict(q=None), dict(exp=None),
                                 dict(out=None), dict(work=None), dict(q=4 * ADDR + 8), dict(out=ADDR + 8),
                                 dict(work=ADDR + 128), dict(exp=ADDR + 2), dict(q_stride=126), dict(q_stride=129),
                                 dict(heads=3), dict(heads=0), dict(heads=65538), dict(out=4 * ADDR + 32),
                                 dict(window=0)], ids=str)
def test_wrong_window_calls_are_refused(ck, bad):
    if bad == dict(window=0):
        bad = dict(window=window(ck, 4, 0))
    assert call(ck, "ck_paged_window_attention", window_args(ck), **bad) == 10


def test_window_scratch_is_refused_for_wrong_arguments(ck):
    n = ctypes.c_size_t()
    L, good = ck.lib(), (ctypes.byref(cache(ck)), ctypes.byref(batch(ck)), 4, ctypes.byref(window(ck)), ctypes.byref(n))
    for i, wrong in ((0, None), (1, None), (2, 3), (3, ctypes.byref(window(ck, 0, 0))), (4, None)):
        assert L.ck_paged_window_attention_work(*good[:i], wrong, *good[i + 1:]) == 10
    assert L.ck_turn_paged_window_work(None, good[0], good[1], good[3], good[4]) == 10
    assert L.ck_turn_paged_window(None, good[0], good[1], good[3], ADDR, 2 * ADDR, 512, 3 * ADDR, 2**40, None) == 10


def advance_args(ck):
    return dict(cache=cache(ck, dev_k=40 * ADDR, dev_v=41 * ADDR), seqs=3, len_in=ADDR, table_in=2 * ADDR, new=3 * ADDR,
                stride=4, window=window(ck), held=4 * ADDR, rows=6, len_out=5 * ADDR, table_out=6 * ADDR, start=7 * ADDR,
                slot=8 * ADDR, position=9 * ADDR, status=10 * ADDR, work=16 * ADDR, work_len=2**20, stream=None)


@pytest.mark.parametrize("bad", [
    dict(cache=None), dict(seqs=0), dict(seqs=65537), dict(len_in=None), dict(table_in=None), dict(new=None),
    dict(stride=0), dict(stride=2**17 + 1), dict(window="empty"), dict(rows=0), dict(rows=2**20 + 1), dict(len_out=None),
    dict(table_out=None), dict(start=None), dict(slot=None), dict(position=None), dict(status=None), dict(work=None),
    dict(work=16 * ADDR + 128), dict(slot=8 * ADDR + 4), dict(position=9 * ADDR + 2), dict(len_in=ADDR + 2),
    # outputs on inputs, on one another, on the pools and on the scratch
    dict(len_out=ADDR), dict(table_out=2 * ADDR + 44), dict(start=3 * ADDR - 12), dict(status=4 * ADDR + 4),
    dict(slot=5 * ADDR - 40), dict(position=6 * ADDR + 44), dict(start=10 * ADDR + 8), dict(status=40 * ADDR + 64),
    dict(slot=41 * ADDR), dict(work=8 * ADDR), dict(work=40 * ADDR), dict(len_out=16 * ADDR + 512)], ids=str)
def test_wrong_steps_of_the_tables_are_refused(ck, bad):
    if bad == dict(window="empty"):
        bad = dict(window=window(ck, 4, 0))
    assert call(ck, "ck_pages_advance", advance_args(ck), **bad) == 10


def test_short_scratch_of_a_step_is_refused(ck):
    n = ctypes.c_size_t()
    assert ck.lib().ck_pages_work(ctypes.byref(cache(ck)), 3, 4, ctypes.byref(n)) == 0
    assert call(ck, "ck_pages_advance", advance_args(ck), work_len=n.value - 1) == 4


def sample_args():
    return dict(logits=ADDR, stride=512, rows=3, vocab=512, temperature=2 * ADDR, top_k=3 * ADDR, top_p=4 * ADDR,
                min_p=5 * ADDR, random=6 * ADDR, exp=7 * ADDR, token=8 * ADDR, prob=9 * ADDR, kept=10 * ADDR, stream=None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(logits=ADDR + 4), dict(stride=511), dict(stride=2**40), dict(rows=0), dict(rows=65537),
    dict(vocab=0), dict(vocab=2**20 + 1, stride=2**21), dict(temperature=None), dict(temperature=2 * ADDR + 1),
    dict(top_k=3 * ADDR + 2), dict(top_p=4 * ADDR + 2), dict(min_p=5 * ADDR + 1), dict(random=None),
    dict(random=6 * ADDR + 4), dict(exp=None), dict(exp=7 * ADDR + 2), dict(token=None), dict(prob=None), dict(kept=None),
    dict(token=8 * ADDR + 2), dict(token=ADDR + 4096), dict(prob=2 * ADDR + 8), dict(kept=3 * ADDR), dict(token=4 * ADDR),
    dict(prob=5 * ADDR - 8), dict(kept=6 * ADDR + 16), dict(token=7 * ADDR + 16384), dict(prob=8 * ADDR + 8),
    dict(kept=9 * ADDR - 8)], ids=str)
def test_wrong_samplings_are_refused(ck, bad):
    assert call(ck, "ck_sample", sample_args(), **bad) == 10


def test_the_place_in_the_table_is_the_floored_quotient(ck):
    """At every temperature's ends of places: floor(256 d / t) below 16 t, 4096 from there."""
    rng = np.random.default_rng(5)
    temperatures = [1, 2, 3, 5, 255, 256, 257, 4095, 65535, 65536, 65537, 98304, 2**20 - 1, 2**20]
    temperatures += [int(t) for t in rng.integers(1, 2**20, 200)]
    for t in temperatures:
        places = np.concatenate([np.arange(0, 4097, 97), [1, 2, 4094, 4095, 4096], rng.integers(0, 4096, 50)])
        first = [-(-int(b) * t // 256) for b in places]
        for d in {x + o for x in first for o in (-1, 0, 1)} | {0, 16 * t - 1, 16 * t, 16 * t + 1, 2**32 - 1}:
            if d >= 0:
                assert ck.host_sample_place(d, t) == (4096 if d >= 16 * t else 256 * d // t), (d, t)


def test_numbers_of_a_window_past_32_bits_are_refused(ck):
    for bad in ((2**32, 5), (-1, 5), (4, 2**32), (4, -1)):
        with pytest.raises(ValueError, match="sinks|window"):
            ck.paged._window(ck.Window(*bad))
        with pytest.raises(ValueError, match="sinks|window"):
            ck.paged._windows(ck.Window(*bad), 3)
    for wrong in ([ck.Window(0, 4)] * 2, (0, 4), [], [4, 4, 4], [ck.Window(0, 4), None, ck.Window(0, 4)]):
        with pytest.raises(ValueError, match="3 layers"):
            ck.paged._windows(wrong, 3)
    assert ck.paged._window(None) is None and ck.paged._windows(None, 3) is None
    each = ck.paged._windows([ck.Window(0, 4), ck.Window(2, 9), ck.Window(1, 1)], 3)
    assert [(w.sinks, w.window) for w in each] == [(0, 4), (2, 9), (1, 1)]


@pytest.mark.parametrize("bad", [
    dict(cache=None), dict(rows_in=0), dict(rows=65537), dict(stride=0), dict(len_in=None), dict(table_in=None),
    dict(parent=None), dict(grow=None), dict(len_out=None), dict(table_out=None), dict(status=None), dict(work=None),
    dict(table_out=2 * ADDR + 60), dict(len_out=ADDR), dict(status=5 * ADDR), dict(held=8 * ADDR), dict(window="empty"),
    dict(work_len=64)], ids=str)
def test_wrong_forks_of_streams_are_refused(ck, bad):
    args = {}
    for name, value in fork_args(ck).items():
        if name == "held":
            args["window"] = window(ck)
        args[name] = value
    if bad == dict(window="empty"):
        bad = dict(window=window(ck, 4, 0))
    assert call(ck, "ck_pages_window_fork", args, **bad) == (4 if "work_len" in bad else 10)


@pytest.mark.parametrize("bad", [
    dict(cache=None), dict(rows=0), dict(stride=2**17 + 1), dict(len=None), dict(table_in=None), dict(table_out=None),
    dict(used=None), dict(status=None), dict(work=None), dict(table_out=2 * ADDR), dict(window="empty"), dict(work_len=64)],
    ids=str)
def test_wrong_packings_of_streams_are_refused(ck, bad):
    args = {}
    for name, value in compact_args(ck).items():
        if name == "table_out":
            args["window"] = window(ck)
        args[name] = value
    if bad == dict(window="empty"):
        bad = dict(window=window(ck, 4, 0))
    assert call(ck, "ck_pages_window_compact", args, **bad) == (4 if "work_len" in bad else 10)


CLUSTERS = (304, 152, 76, 38)


def window_plan(ck, view, seqs, new, length, heads, kv_heads, hd, page=16, rows=None):
    """The kernel (0 a few queries, 1 tiles, 2 single rows) and the scratch of a call with a window (None:
    without) on a device of 152 multiprocessors."""
    kernel, work = ctypes.c_uint32(), ctypes.c_size_t()
    c = cache(ck, kv_heads=kv_heads, page=page, head_dim=hd)
    b = batch(ck, seqs=seqs, rows=rows or seqs * new, stride=2**17, max_new=new, max_len=length)
    w = None if view is None else ctypes.byref(window(ck, *view))
    rc = ck.lib().ck_host_window_attention_plan(ctypes.byref(c), ctypes.byref(b), heads, w, 152, 232448,
                                                (ctypes.c_int32 * 4)(*CLUSTERS), ctypes.byref(kernel), ctypes.byref(work))
    assert rc == 0
    return kernel.value, work.value


PLANS = [(1, 1, 8192, 32, 32, 64), (64, 1, 8192, 32, 8, 32), (2, 201, 2047, 32, 32, 128), (1, 256, 7936, 32, 32, 64),
         (1, 2048, 8192, 32, 32, 32), (8, 512, 32768, 32, 8, 16), (4096, 1, 32768, 32, 32, 32), (3, 40, 900, 8, 2, 8),
         (1, 1, 130001, 4, 1, 4)]


@pytest.mark.parametrize("shape", PLANS, ids=str)
def test_a_window_that_holds_everything_plans_as_the_whole_cache(ck, shape):
    length = shape[2]
    whole = window_plan(ck, None, *shape)
    for view in ((0, length), (length, 1), (2**32 - 1, 2**32 - 1), (7, 2**32 - 1)):
        assert window_plan(ck, view, *shape) == whole


@pytest.mark.parametrize("seqs,new,length,heads,kv,hd", PLANS)
@pytest.mark.parametrize("sinks,size", [(0, 1), (4, 100), (5, 511), (70, 700), (4, 4000), (0, 30000), (9, 120000)])
def test_the_scratch_of_a_window_holds_the_places_that_are_seen(ck, seqs, new, length, heads, kv, hd, sinks, size):
    """A few queries: none, or the scores of every query's places, up to 2 GB of them at a time.  Tiles: the
    scores of 128 rows' places and the sums of every cluster, of one of the sizes.  Single rows: a row's places."""
    kernel, work = window_plan(ck, (sinks, size), seqs, new, length, heads, kv, hd)
    group = heads // kv
    places = min(length, sinks + size)
    if kernel == 0:
        assert 256 <= work <= 2**31
        scores = 8 * seqs * heads * new * places
        assert work == 256 or work >= min(scores, 2**30)
        # 227 KB of shared memory hold no more than this of up to four queries, of sixteen blocks
        if 8 * places * min(4, new * group) > 16 * 232448:
            assert work > 256
    elif kernel == 1:
        tiles = seqs * kv * -(-new * group // 128)
        places = min(length, sinks + size + min(new - 1, 127 // group))
        sizes = [min(tiles, n) * (4 * 128 * places + 8 * 128 * hd * 2**i) for i, n in enumerate(CLUSTERS)]
        assert hd >= 64 and work >= min(sizes)
    else:
        assert work >= 8 * places
    # a window takes no more than the whole cache does through the same kernel
    other, most = window_plan(ck, None, seqs, new, length, heads, kv, hd)
    if kernel == other == 0 and work > 256 and most > 256:
        assert work <= max(most, 2**31)


def test_windows_whose_scores_take_several_launches(ck):
    """Two gigabytes at a time where all would be more; single rows where the launches would be too many."""
    for shape in ((2, 300, 20500, 32, 8, 4), (1, 500, 20500, 32, 8, 4)):
        kernel, work = window_plan(ck, (3, 19999), *shape)
        seqs, new, _, heads = shape[:4]
        assert kernel == 0 and 2**30 < work <= 2**31 < 8 * seqs * heads * new * 20000
    kernel, work = window_plan(ck, (0, 2**19), 65535, 1000, 2**20 - 1, 32, 32, 32, page=256, rows=70000)
    assert kernel == 2 and 8 * 2**19 <= work <= 4 * 152 * 8 * (2**19 + 16)


def test_wrong_arguments_of_a_window_plan_are_refused(ck):
    kernel, work, n = ctypes.c_uint32(), ctypes.c_size_t(), (ctypes.c_int32 * 4)(1, 1, 1, 1)
    good = dict(cache=cache(ck), batch=batch(ck), heads=4, window=window(ck), sms=152, smem=232448, clusters=n,
                kernel=ctypes.byref(kernel), work=ctypes.byref(work))
    assert call(ck, "ck_host_window_attention_plan", good) == 0
    for bad in (dict(cache=None), dict(batch=None), dict(heads=3), dict(sms=0), dict(smem=2**21), dict(clusters=None),
                dict(kernel=None), dict(work=None), dict(window=window(ck, 4, 0))):
        assert call(ck, "ck_host_window_attention_plan", good, **bad) == 10
