"""What the paged cache's operators and beam search refuse, and their host routines: no GPU
needed (every refusal is decided from the arguments alone, before any device call)."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def ck():
    import fixed_point_int8_gb300 as ck
    from fixed_point_int8_gb300 import build
    build.build()
    return ck


def plain_log_sum(z):
    z = max(z, 2**30)
    n = z.bit_length() - 31
    y = z >> n
    t = ((y - 2**30) << 30) // (y + 2**30)
    square, c = (t * t) >> 30, 0
    for i in range(7, -1, -1):
        c = (2**31 // (2 * i + 1) + 1) // 2 + ((c * square) >> 30)
    return (n * 744261118 + 2 * ((t * c) >> 30) + 2**13) >> 14


def test_log_sum_is_the_logarithm(ck):
    """The integer series against its definition and against the real logarithm: y is cut to 30
    fraction bits (2^-30 relative), each of at most 16 cut products loses below 2^-30, the series
    after t^15 leaves t^17 / 17 * 2 * 9/8 < 2^-29, and the last step rounds to half of 2^-16."""
    rng = np.random.default_rng(1)
    zs = [0, 1, 2**30 - 1, 2**30, 2**30 + 1, 2**31 - 1, 2**31, 2**50, 2**50 - 1, 2**52]
    zs += [2**int(e) + int(r) for e, r in zip(rng.integers(30, 51, 2000), rng.integers(0, 2**30, 2000))]
    for z in zs:
        got = ck.host_log_sum(z)
        assert got == plain_log_sum(z), z
        real = math.log(max(z, 2**30) / 2**30)
        assert abs(got / 2**16 - real) <= 2**-17 + 40 * 2**-30, z


ADDR = 1 << 20  # stands for an aligned device address: nothing reads it


def call(ck, name, good, **changed):
    args = dict(good)  # (structures are passed by their addresses)
    for key, value in changed.items():
        assert key in args
        args[key] = value
    return getattr(ck.lib(), name)(*(ctypes.byref(a) if isinstance(a, ctypes.Structure) else a for a in args.values()))


def cache(ck, **changed):
    f = dict(dev_k=ADDR, dev_v=2 * ADDR, pages=8, layers=2, kv_heads=2, page=16, head_dim=32)
    f.update(changed)
    return ck.paged._Cache(*f.values())


def batch(ck, **changed):
    f = dict(dev_start=ADDR, dev_len=ADDR, dev_table=ADDR, dev_status=ADDR, seqs=3, rows=6, stride=4, max_new=2,
             max_len=64)
    f.update(changed)
    return ck.paged._Batch(*f.values())


BAD_CACHES = [dict(dev_k=None), dict(dev_v=None), dict(dev_k=ADDR + 8), dict(dev_v=ADDR + 4), dict(pages=0),
              dict(pages=2**24 + 1), dict(layers=0), dict(layers=4096), dict(kv_heads=0), dict(kv_heads=4097),
              dict(page=4), dict(page=24), dict(page=512), dict(head_dim=2), dict(head_dim=48), dict(head_dim=256)]
BAD_BATCHES = [dict(dev_start=None), dict(dev_len=None), dict(dev_table=None), dict(dev_status=None),
               dict(dev_status=ADDR + 4), dict(dev_table=ADDR + 2), dict(seqs=0), dict(seqs=65536), dict(rows=0),
               dict(rows=2**20 + 1), dict(stride=0), dict(stride=2**17 + 1), dict(max_new=0), dict(max_new=7),
               dict(max_len=0), dict(max_len=2**20)]


def store_args(ck):
    return dict(cache=cache(ck), layer=1, batch=batch(ck), q=4 * ADDR, q_stride=128, k=5 * ADDR, k_stride=64,
                v=6 * ADDR, v_stride=64, heads=4, rope=7 * ADDR, rope_rows=64, rot=32, half=0, out=8 * ADDR, stream=None)


def attention_args(ck):
    return dict(cache=cache(ck), layer=1, batch=batch(ck), q=4 * ADDR, q_stride=128, heads=4, exp=ADDR, inv=1,
                out=8 * ADDR, work=16 * ADDR, work_len=2**40, stream=None)


@pytest.mark.parametrize("bad", BAD_CACHES + BAD_BATCHES, ids=str)
def test_wrong_caches_and_batches_are_refused(ck, bad):
    key = "cache" if bad.keys() & {n for n, _ in ck.paged._Cache._fields_} else "batch"
    value = cache(ck, **bad) if key == "cache" else batch(ck, **bad)
    assert call(ck, "ck_paged_store", store_args(ck), **{key: value}) == 10
    assert call(ck, "ck_paged_attention", attention_args(ck), **{key: value}) == 10


@pytest.mark.parametrize("bad", [dict(cache=None), dict(layer=2), dict(batch=None), dict(q=None), dict(k=None),
                                 dict(v=None), dict(rope=None), dict(out=None), dict(q=4 * ADDR + 8),
                                 dict(out=8 * ADDR + 8), dict(rope=ADDR + 8), dict(q_stride=126), dict(q_stride=129),
                                 dict(k_stride=62), dict(v_stride=65), dict(heads=0), dict(heads=65537),
                                 dict(rope_rows=0), dict(rot=6), dict(rot=36), dict(q_stride=2**40),
                                 dict(out=4 * ADDR), dict(out=5 * ADDR + 16), dict(out=6 * ADDR - 16)], ids=str)
def test_wrong_stores_are_refused(ck, bad):
    assert call(ck, "ck_paged_store", store_args(ck), **bad) == 10


@pytest.mark.parametrize("bad", [dict(cache=None), dict(layer=2), dict(batch=None), dict(q=None), dict(exp=None),
                                 dict(out=None), dict(work=None), dict(q=4 * ADDR + 8), dict(out=ADDR + 8),
                                 dict(work=ADDR + 128), dict(exp=ADDR + 2), dict(q_stride=126), dict(q_stride=129),
                                 dict(heads=3), dict(heads=0), dict(heads=65538), dict(out=4 * ADDR + 32)], ids=str)
def test_wrong_attention_calls_are_refused(ck, bad):
    assert call(ck, "ck_paged_attention", attention_args(ck), **bad) == 10


def test_work_sizes_are_refused_for_wrong_arguments(ck):
    n = ctypes.c_size_t()
    out = ctypes.byref(n)
    L = ck.lib()
    assert L.ck_pages_work(ctypes.byref(cache(ck)), 4, 4, None) == 10
    for c, rows, stride in ((cache(ck, page=7), 4, 4), (cache(ck), 0, 4), (cache(ck), 65537, 4), (cache(ck), 4, 0),
                            (cache(ck), 4, 2**17 + 1), (None, 4, 4)):
        assert L.ck_pages_work(c and ctypes.byref(c), rows, stride, out) == 10
    assert L.ck_pages_work(ctypes.byref(cache(ck)), 4, 4, out) == 0 and n.value > 0
    for groups, beams, vocab in ((0, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, 0), (1, 1, 2**20 + 1), (1025, 64, 9)):
        assert L.ck_beam_work(groups, beams, vocab, out) == 10
    assert L.ck_beam_work(1, 1, 1, None) == 10
    assert L.ck_beam_work(1024, 64, 9, out) == 0 and n.value > 0
    assert L.ck_paged_attention_work(ctypes.byref(cache(ck)), ctypes.byref(batch(ck)), 3, out) == 10
    assert L.ck_paged_attention_work(ctypes.byref(cache(ck)), ctypes.byref(batch(ck)), 4, None) == 10


def fork_args(ck):
    return dict(cache=cache(ck), rows_in=4, len_in=ADDR, table_in=2 * ADDR, rows=4, parent=3 * ADDR, grow=4 * ADDR,
                stride=4, held=None, len_out=5 * ADDR, table_out=6 * ADDR, status=7 * ADDR, work=8 * ADDR,
                work_len=ADDR, stream=None)


@pytest.mark.parametrize("bad", [dict(cache=None), dict(rows_in=0), dict(rows=0), dict(rows_in=65537), dict(rows=65537),
                                 dict(stride=0), dict(stride=2**17 + 1), dict(len_in=None), dict(table_in=None),
                                 dict(parent=None), dict(grow=None), dict(len_out=None), dict(table_out=None),
                                 dict(status=None), dict(work=None), dict(work=8 * ADDR + 4), dict(table_out=2 * ADDR),
                                 dict(table_out=2 * ADDR + 60), dict(len_out=ADDR), dict(status=5 * ADDR),
                                 dict(len_out=8 * ADDR), dict(parent=ADDR + 2), dict(held=8 * ADDR)], ids=str)
def test_wrong_forks_are_refused(ck, bad):
    assert call(ck, "ck_pages_fork", fork_args(ck), **bad) == 10


def test_short_scratch_is_refused(ck):
    assert call(ck, "ck_pages_fork", fork_args(ck), work_len=64) == 4
    assert call(ck, "ck_pages_compact", compact_args(ck), work_len=64) == 4
    assert call(ck, "ck_beam_select", beam_args(ck), work_len=64) == 4


def compact_args(ck):
    return dict(cache=cache(ck), rows=4, len=ADDR, table_in=2 * ADDR, stride=4, table_out=3 * ADDR, used=4 * ADDR,
                status=5 * ADDR, work=8 * ADDR, work_len=ADDR, stream=None)


@pytest.mark.parametrize("bad", [dict(cache=None), dict(rows=0), dict(rows=65537), dict(len=None), dict(table_in=None),
                                 dict(stride=0), dict(table_out=None), dict(used=None), dict(status=None),
                                 dict(work=None), dict(work=ADDR * 8 + 16), dict(table_out=2 * ADDR + 4),
                                 dict(used=3 * ADDR), dict(status=ADDR)], ids=str)
def test_wrong_packings_are_refused(ck, bad):
    assert call(ck, "ck_pages_compact", compact_args(ck), **bad) == 10


def beam_args(ck):
    return dict(logits=ADDR, stride=100, groups=2, beams=4, vocab=100, scores=2 * ADDR, done=3 * ADDR, exp=4 * ADDR,
                flags=1, done_token=2, scores_out=5 * ADDR, parent=6 * ADDR, token=7 * ADDR, done_out=8 * ADDR,
                work=9 * ADDR, work_len=ADDR, stream=None)


@pytest.mark.parametrize("bad", [dict(logits=None), dict(logits=ADDR + 4), dict(stride=99), dict(groups=0), dict(beams=0),
                                 dict(beams=65), dict(vocab=0), dict(scores=None), dict(done=None), dict(exp=None),
                                 dict(flags=2), dict(done_token=100), dict(scores_out=None), dict(parent=None),
                                 dict(token=None), dict(done_out=None), dict(work=None), dict(scores_out=2 * ADDR),
                                 dict(done_out=3 * ADDR), dict(token=6 * ADDR + 4), dict(scores_out=ADDR + 8)], ids=str)
def test_wrong_selections_are_refused(ck, bad):
    assert call(ck, "ck_beam_select", beam_args(ck), **bad) == 10


def test_paged_turns_and_tables_without_a_model_are_refused(ck):
    L, n, p = ck.lib(), ctypes.c_size_t(), ctypes.c_void_p()
    c, b = ctypes.byref(cache(ck)), ctypes.byref(batch(ck))
    assert L.ck_turn_paged_work(None, c, b, ctypes.byref(n)) == 10
    assert L.ck_turn_paged(None, c, b, ADDR, ADDR, 64, ADDR, 1 << 30, None) == 10
    assert L.ck_model_tables(None, ctypes.byref(p), ctypes.byref(p), ctypes.byref(ctypes.c_uint32())) == 10


def test_the_binding_checks_tensors(ck):
    """Types, shapes, strides and devices that the library cannot see."""
    import torch
    pool = torch.zeros(3, 1, 2, 8, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ck.PagedCache(pool, pool)                                   # not on a CUDA device
    with pytest.raises(ValueError):
        ck.PagedCache(pool[0], pool[0])
    with pytest.raises(ValueError):
        ck.PagedCache(pool.long(), pool.long())
    with pytest.raises(ValueError):
        ck.PagedBatch(torch.zeros(2, 3, dtype=torch.int64), pool, pool, None, 1, 1, 1)
    for t, rows in ((torch.zeros(2, 3), 2), (torch.zeros(2, 3, dtype=torch.int64), 3),
                    (torch.zeros(3, 2, dtype=torch.int64).t(), 2)):
        with pytest.raises(ValueError):
            ck.paged._check_rows("q", t, rows, 0)


def attention_plan(ck, seqs, new, length, heads, kv_heads, hd, clusters, page=16, sms=152, smem=232448, rows=None):
    """The kernel (0 a few queries, 1 tiles, 2 single rows) and the scratch of a call on a device."""
    kernel, work = ctypes.c_uint32(), ctypes.c_size_t()
    c = cache(ck, kv_heads=kv_heads, page=page, head_dim=hd)
    b = batch(ck, seqs=seqs, rows=rows or seqs * new, stride=2**17, max_new=new, max_len=length)
    rc = ck.lib().ck_host_attention_plan(ctypes.byref(c), ctypes.byref(b), heads, sms, smem, (ctypes.c_int32 * 4)(*clusters),
                                         ctypes.byref(kernel), ctypes.byref(work))
    assert rc == 0
    return kernel.value, work.value


@pytest.mark.parametrize("hd,new,length,heads,kv", [(64, 256, 7936, 32, 32), (128, 201, 2047, 32, 32), (64, 70, 600, 32, 4)])
@pytest.mark.parametrize("clusters", [(304, 152, 76, 38), (304, -1, -1, -1), (304, 152, -1, 38), (-1, -1, 76, 38),
                                      (304, 0, 0, 0), (-1, 152, 0, -1), (0, 0, 0, 0), (-1, -1, -1, -1)], ids=str)
def test_a_plan_is_whole_whatever_the_device_answers(ck, hd, new, length, heads, kv, clusters):
    """A lookup of resident clusters that fails takes that cluster size out of the choice and no more:
    tiles always come with the scratch of every block that runs."""
    kernel, work = attention_plan(ck, 1, new, length, heads, kv, hd, clusters)
    assert (kernel, work) == attention_plan(ck, 1, new, length, heads, kv, hd, [max(n, 0) for n in clusters])
    tiles = kv * -(-new * (heads // kv) // 128)
    if max(clusters) <= 0:
        assert kernel != 1 and work >= 256
    else:
        # of one cluster size: 128 rows' scores of all positions a cluster (the positions split over its
        # blocks), and 128 rows' sums of 64 bits a block
        sizes = [min(tiles, n) * (4 * 128 * length + 8 * 128 * hd * 2**i) for i, n in enumerate(clusters) if n > 0]
        assert kernel == 1 and work >= min(sizes)


def test_wrong_arguments_of_a_plan_are_refused(ck):
    kernel, work, n = ctypes.c_uint32(), ctypes.c_size_t(), (ctypes.c_int32 * 4)(1, 1, 1, 1)
    good = dict(cache=cache(ck), batch=batch(ck), heads=4, sms=152, smem=232448, clusters=n, kernel=ctypes.byref(kernel),
                work=ctypes.byref(work))
    assert call(ck, "ck_host_attention_plan", good) == 0
    for bad in (dict(cache=None), dict(batch=None), dict(heads=3), dict(heads=0), dict(sms=0), dict(smem=2**21),
                dict(clusters=None), dict(kernel=None), dict(work=None), dict(cache=cache(ck, page=7)),
                dict(batch=batch(ck, seqs=0))):
        assert call(ck, "ck_host_attention_plan", good, **bad) == 10


@pytest.mark.parametrize("seqs,new,length,heads,kv,hd", [(1, 2048, 8192, 32, 32, 32), (1, 4096, 8192, 32, 32, 32),
                                                         (8, 512, 32768, 32, 8, 16), (256, 1, 32768, 32, 32, 64),
                                                         (4096, 1, 32768, 32, 32, 32), (1, 2, 8192, 4, 4, 4)])
def test_the_scratch_of_a_few_queries_is_bounded(ck, seqs, new, length, heads, kv, hd):
    """Scores that do not fit shared memory: no more than 2 GB of them at once, whatever the batch."""
    kernel, work = attention_plan(ck, seqs, new, length, heads, kv, hd, (304, 152, 76, 38))
    assert kernel == 0 and 256 <= work <= 2**31


def test_bounds_that_would_take_very_many_launches_go_to_single_rows(ck):
    """2^16 sequences of up to 2^20 positions by their bounds, 70,000 rows in all."""
    kernel, work = attention_plan(ck, 65535, 1000, 2**20 - 1, 32, 32, 32, (304, 152, 76, 38), page=256, rows=70000)
    assert kernel == 2 and work <= 4 * 152 * 8 * 2**20


def test_numbers_past_32_bits_are_refused(ck):
    """A number that ctypes would cut to 32 bits (here: to a good one) is an error."""
    import torch

    class Pool:
        k = torch.zeros(1)
        _struct = cache(ck)
        _c = ctypes.addressof(_struct)

    assert ck.PagePlan(Pool, 4, 4).rows == 4
    for rows, stride in ((2**32 + 4, 4), (4, 2**32 + 4), (-2**32 + 4, 4), (4, -1)):
        with pytest.raises(ValueError):
            ck.PagePlan(Pool, rows, stride)
    for sizes in ((2**32 + 1, 1, 5), (1, 2**32 + 1, 5), (1, 1, 2**32 + 5), (-1, 1, 5)):
        with pytest.raises(ValueError):
            ck.BeamPlan(*sizes)
    with pytest.raises(ValueError):
        ck.set_beam_wait_limit(2**32)
    with pytest.raises(TypeError):
        ck.PagePlan(Pool, 4.0, 4)
    assert ck.PagePlan(Pool, np.int64(4), np.uint8(4)).stride == 4


def test_a_stream_of_another_device_is_refused(ck, monkeypatch):
    """Its number on the current device could be any stream's, the default one's among them."""
    import torch

    class On:
        cuda_stream = 0

        def __init__(self, index):
            self.device = torch.device("cuda", index)

    class Here:
        device, _c = 0, None

    monkeypatch.setattr(ck.paged, "_device", lambda: 0)
    assert ck.paged._devices(Here, Here, None) == ck.paged._devices(Here, Here, On(0)) == 0
    for call_it in (lambda: ck.paged._devices(Here, Here, On(1)), lambda: ck.paged_attention_work(Here, Here, 1, stream=On(1)),
                    lambda: ck.paged_attention(Here, 0, Here, None, None, 1, stream=On(1)),
                    lambda: ck.paged_store(Here, 0, Here, None, None, None, None, stream=On(1)),
                    lambda: ck.paged.turn_paged(None, Here, Here, None, stream=On(1)),
                    lambda: ck.paged.turn_paged_work(None, Here, Here, stream=On(1))):
        with pytest.raises(ValueError, match="stream"):
            call_it()
    there = Here()
    there.device = 1
    with pytest.raises(ValueError, match="current CUDA device"):
        ck.paged_attention_work(there, Here, 1)


POOL = 8 * 2 * 2 * 16 * 32 * 4     # bytes of either pool of cache()


def apart(ck):
    """The batch's arrays at places of their own: 16 bytes of starts, 12 of lengths, 48 of the table, 24 of
    status words."""
    return batch(ck, dev_start=20 * ADDR, dev_len=21 * ADDR, dev_table=22 * ADDR, dev_status=23 * ADDR)


@pytest.mark.parametrize("at,size", [(ADDR, POOL), (2 * ADDR, POOL), (20 * ADDR, 16), (21 * ADDR, 12), (22 * ADDR, 48),
                                     (23 * ADDR, 24), (4 * ADDR, 6 * 128 * 8)])
def test_outputs_on_inputs_are_refused(ck, at, size):
    """Outputs and scratch that begin on an input's last bytes or end on its first ones."""
    last = (at + size - 1) // 16 * 16
    rows = 6 * 128 * 8
    assert call(ck, "ck_paged_store", store_args(ck), batch=apart(ck), out=last) == 10
    assert call(ck, "ck_paged_store", store_args(ck), batch=apart(ck), out=at - rows + 16) == 10
    good = dict(batch=apart(ck), exp=24 * ADDR, work=16 * ADDR, work_len=ADDR)
    for bad in (dict(out=last), dict(out=at - rows + 16), dict(work=(at + size - 1) // 256 * 256),
                dict(work=at - 512, work_len=513)):
        assert call(ck, "ck_paged_attention", attention_args(ck), **{**good, **bad}) == 10


def test_outputs_on_tables_and_scratch_are_refused(ck):
    assert call(ck, "ck_paged_store", store_args(ck), batch=apart(ck), out=7 * ADDR + 64 * 32 * 4 - 16) == 10
    good = dict(batch=apart(ck), exp=24 * ADDR, work=16 * ADDR, work_len=ADDR)
    for bad in (dict(out=24 * ADDR + 4096 * 4), dict(work=24 * ADDR + 16384), dict(out=17 * ADDR - 16),
                dict(out=16 * ADDR - 6 * 128 * 8 + 16)):
        assert call(ck, "ck_paged_attention", attention_args(ck), **{**good, **bad}) == 10


def test_tables_on_pools_and_selections_on_the_exponentials_are_refused(ck):
    for at in (ADDR, 2 * ADDR):
        for place in (at + POOL - 4, at - 12):
            # (the inputs elsewhere; outputs of 16 bytes and more)
            moved = dict(len_in=30 * ADDR, table_in=31 * ADDR)
            for name in ("len_out", "table_out", "status"):
                assert call(ck, "ck_pages_fork", fork_args(ck), **{**moved, name: place}) == 10
            moved = dict(len=30 * ADDR, table_in=31 * ADDR)
            for name in ("table_out", "status"):
                assert call(ck, "ck_pages_compact", compact_args(ck), **{**moved, name: place}) == 10
        assert call(ck, "ck_pages_compact", compact_args(ck), len=30 * ADDR, table_in=31 * ADDR, used=at + 40) == 10
        work = dict(work=at + POOL - 256)
        assert call(ck, "ck_pages_fork", fork_args(ck), len_in=30 * ADDR, table_in=31 * ADDR, **work) == 10
        assert call(ck, "ck_pages_compact", compact_args(ck), len=30 * ADDR, table_in=31 * ADDR, **work) == 10
    for name in ("scores_out", "parent", "token", "done_out", "work"):
        assert call(ck, "ck_beam_select", beam_args(ck), **{name: 4 * ADDR + 16384}) == 10
