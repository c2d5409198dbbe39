"""Forms of the streams' operators that sizes, settings or a model's shape choose: scores in scratch and in
several launches, passes of models with large heads, tables as long as they go.  All of it is integer
work: tolerance 0."""
import numpy as np
import pytest

import synth
from test_gpu_paged import EXP, Setup, ck, cuda, plain_attention  # noqa: F401
from test_gpu_streams import PlainStream, WINDOW_TILES, Windowed, plain_advance, seen
from test_gpu_stream_tables import i32

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- attention over a window

def some_rows(s, layer, q, inv, out, at):
    """The outputs of some (row, head) pairs against the plain form."""
    for row, h in at:
        i = int(np.searchsorted(s.starts, row, side="right")) - 1
        pos = s.lens[i] - s.news[i] + row - int(s.starts[i])
        t = seen(pos, *s.view)
        c = slice(h * s.hd, (h + 1) * s.hd)
        K, V = (pool[s.table[i, t // s.page], layer, h // (s.heads // s.kv), t % s.page] for pool in (s.k, s.v))
        assert np.array_equal(out[row, c].cpu().numpy(), plain_attention(q[row, c], K, V, inv)), (row, h)


# lens, news, heads, kv heads, head, page, sinks, window: a sequence over sixteen blocks, a block a key head,
# chunks of several groups of queries, two groups of pages of different lengths in a block
@pytest.mark.parametrize("lens,news,heads,kv,hd,page,sinks,window", [
    ([130001, 124000], [1, 1], 4, 1, 4, 64, 5, 120000),
    ([int(n) for n in np.linspace(4100, 8000, 40)], [1] * 40, 32, 8, 8, 16, 4, 4000),
    ([8000, 7001, 6000, 5005, 4000, 3003, 2000, 1000], [20, 19, 1, 7, 20, 3, 0, 13], 8, 8, 4, 8, 33, 4500),
    ([9000, 6100, 4200], [33, 40, 12], 24, 6, 16, 32, 900, 3700),
])
def test_windows_whose_scores_lie_in_the_scratch(ck, lens, news, heads, kv, hd, page, sinks, window):
    """More places than a block has shared memory for, by few queries."""
    import torch
    s = Windowed(ck, lens, news, heads, kv, hd, page, sinks, window, seed=hd, layers=1, lead=1, tail=2)
    work = ck.paged_attention_work(s.cache, s.batch, heads, window=s.view)
    assert work.numel() > 8 * 4 * 4000  # (at least a block's scores; shared memory takes none)
    q, inv = s.queries(2**19), synth.inv_sqrt_head(hd)
    out = torch.full((s.rows, heads * hd), 7, dtype=torch.int64, device="cuda")
    rc, _ = s.run(ck, q, inv, out=out, work=work)
    assert rc == 0 and s.batch.errors() == [None] * len(lens)
    rng = np.random.default_rng(1)
    rows = [int(r) for r in rng.integers(s.starts[0], s.starts[-1], 40)] + [int(s.starts[0]), int(s.starts[-1]) - 1]
    some_rows(s, 0, q, inv, out, [(r, int(rng.integers(heads))) for r in rows] + [(rows[0], h) for h in range(heads)])
    assert (out[:1] == 7).all() and (out[-2:] == 7).all() and not (out[1:-2] == 7).all(1).any()
    rc, again = s.run(ck, q, inv, work=torch.empty(work.numel() - 1, dtype=torch.uint8, device="cuda"))
    assert rc == 4


@pytest.mark.parametrize("lens,news", [([20500, 20300], [300, 280]),  # a launch a sequence
                                       ([20500], [500])])              # two, of groups of queries
def test_windows_in_launches_that_share_the_scratch(ck, lens, news):
    heads, kv, hd = 32, 8, 4
    s = Windowed(ck, lens, news, heads, kv, hd, 32, 3, 19999, seed=len(lens), layers=1)
    assert 2**30 < ck.paged_attention_work(s.cache, s.batch, heads, window=s.view).numel() <= 2**31
    q, inv = s.queries(2**19), synth.inv_sqrt_head(hd)
    rc, out = s.run(ck, q, inv)
    assert rc == 0 and s.batch.errors() == [None] * len(lens)
    rng = np.random.default_rng(2)
    rows = list(range(0, s.rows, 37)) + [int(a) for a in s.starts[1:] - 1] + [int(a) for a in s.starts[:-1]]
    some_rows(s, 0, q, inv, out, [(r, int(rng.integers(heads))) for r in rows])


def test_window_scratch_a_step_too_small(ck):
    import torch
    s = Windowed(ck, [1900, 733], [70, 129], 32, 8, 64, 16, 4, 500)
    n = ck.paged_attention_work(s.cache, s.batch, 32, window=s.view).numel()
    for short in (1, 256, n - 1):
        rc, _ = s.run(ck, s.queries(), 1 << 21, work=torch.empty(n - short, dtype=torch.uint8, device="cuda"))
        assert rc == 4


@pytest.mark.parametrize("lens,news,heads,kv,hd,page", [([300], [1], 3, 3, 128, 256), ([1025], [1], 32, 32, 64, 64),
                                                        ([300, 77, 12], [129, 20, 12], 4, 4, 32, 64)] +
                         [c[:6] for c in WINDOW_TILES[:2]])
def test_a_window_that_misses_one_position(ck, lens, news, heads, kv, hd, page):
    """One position shorter than the longest sequence: its last row misses its first position, and no
    other row anything."""
    import torch
    s = Setup(ck, lens, news, heads, kv, hd, page, seed=2)
    q, exp = (s.rng.standard_normal((s.rows, heads * hd)) * 65536).astype(np.int64), cuda(EXP.view(np.int32))
    assert lens[0] == max(lens) and lens[0] not in lens[1:]
    rc, whole = ck.paged_attention(s.cache, 0, s.batch, cuda(q), exp, 1 << 21)
    assert rc == 0
    rc, out = ck.paged_attention(s.cache, 0, s.batch, cuda(q), exp, 1 << 21, window=ck.Window(0, lens[0] - 1))
    assert rc == 0
    last = int(s.starts[1]) - 1
    keep = torch.arange(s.rows, device="cuda") != last
    assert torch.equal(out[keep], whole[keep])
    t = np.arange(1, lens[0])
    for h in range(heads):
        c = slice(h * hd, (h + 1) * hd)
        K, V = (pool[s.table[0, t // page], 0, h // (heads // kv), t % page] for pool in (s.k, s.v))
        assert np.array_equal(out[last, c].cpu().numpy(), plain_attention(q[last, c], K, V, 1 << 21))
    assert not torch.equal(out[last], whole[last])


# ---------------------------------------------------------------- a model's layers

HUGE = 10**6


@pytest.mark.parametrize("heads,kv,views", [
    (8, 2, [(4, 30), (0, HUGE), (2, 200)]),    # heads of 64: few queries, the whole cache, tiles
    (4, 1, [(2, 200), (4, 30), (0, HUGE)]),    # heads of 128
    (8, 2, [(4, 200), (0, 60), (33, 200)]),    # pages come back
], ids=str)
def test_layers_of_large_heads_whose_windows_take_different_kernels(ck, heads, kv, views):
    """Two chunks of 300 and single tokens through three layers, each with a window (and a scratch) of its
    own: the logits are those of a run from the oracle's steps."""
    hd = 512 // heads
    spec = synth.ModelSpec("streams", 512, 352, 3, heads, kv, 512, 1024, tied=False, seed=0x5EED0078)
    art = synth.build_artifact(spec)
    rc, model = ck.Model.load(art)
    assert rc == 0
    whole = any(w == HUGE for _, w in views)
    widest = None if whole else ck.Window(max(s for s, _ in views), max(w for _, w in views))
    windows, page, steps = [ck.Window(*v) for v in views], 16, [300, 300, 1, 1]
    pages = 40 if whole else 36
    cache = ck.PagedCache.empty(pages, spec.layers, kv, page, hd)
    plan, lens, table = ck.PagePlan(cache, 1, 40), i32([0]), i32([[-1] * 40])
    ids = [int(t) for t in synth.prompt_ids(spec, sum(steps))]
    plain, done = PlainStream(spec, art, views), 0
    for n in steps:
        rc, got = plan.advance(lens, table, i32([n]), n, window=widest)
        assert rc == 0 and got.status.tolist() == [0]
        lens, table = got.lens, got.table
        batch = ck.PagedBatch(table, lens, got.starts, None, n, n, done + n)
        each = [ck.paged_attention_work(cache, batch, heads, window=w).numel() for w in windows]
        if n > 1 and done == 300:
            assert [e > 1 << 20 for e in each] == [w >= 200 for _, w in views]  # the tiles
        work = model.turn_paged_work(cache, batch, window=windows)
        assert work.numel() >= max(each)
        rc, logits = model.turn_paged(cache, batch, i32(ids[done:done + n]), work=work, window=windows)
        assert rc == 0 and batch.errors() == [None]
        want = [plain.logits(t, done + i) for i, t in enumerate(ids[done:done + n])][-1]
        assert np.array_equal(logits[0].cpu().numpy(), want), done
        done += n
    if not whole:
        assert (table == -1).sum() > 16


# ---------------------------------------------------------------- long tables

@pytest.mark.parametrize("seqs,stride,page,view", [(1, 8192, 16, None), (1, 8192, 16, (4, 1000)), (3, 8192, 8, (9000, 70)),
                                                   (1, 131072, 8, (5, 1024)), (1, 131072, 8, None), (9, 131072, 16, (40, 1000))])
def test_steps_of_long_tables(ck, seqs, stride, page, view):
    """Tables of thousands of entries, a few sequences: one block, a cluster, and four kernels; up to 2^20
    - 1 positions, which and not the table is the bound of the longest."""
    rng = np.random.default_rng(stride + seqs)
    view = view and ck.Window(*view)
    most = min(stride * page, 2**20 - 1)
    pages = 160_000  # (above what is kept and asked for)
    lens = [int(n) for n in rng.integers(most - 40_000, most, seqs)]
    table = np.full((seqs, stride), -1, np.int64)
    ids, at = rng.permutation(pages), 0
    for s, n in enumerate(lens):
        for i in range(-(-n // page)):
            if view is None or i * page < view.sinks or n - ((i + 1) * page - 1) < view.window:
                table[s, i] = ids[at]
                at += 1
    plan = ck.PagePlan(ck.PagedCache.empty(pages, 1, 1, page, 4), seqs, stride)
    table = table.tolist()
    for turn in range(3):
        # to the bound, at it, and past it
        ask = [[most - n if s == 0 else 17, 0 if s == 0 else 5, 1][turn] for s, n in enumerate(lens)]
        rc, got = plan.advance(i32(lens), i32(table), i32(ask), 50_000, window=view)
        assert rc == 0
        want = plain_advance(lens, table, ask, 50_000, page, pages, view)
        for name, a, b in zip(got._fields, got, want):
            assert a.tolist() == b, (name, turn)
        assert want[5][0] == (7 if turn == 2 else 0) and want[1][0] == most
        table, lens = want[0], want[1]


def test_lengths_at_the_bound_of_positions(ck):
    """2^20 - 1 positions, where the table would hold twice as many."""
    page, stride, view = 16, 2**17, (0, 20)
    table = [[-1] * stride for _ in range(5)]
    for s in range(5):
        for i in range(65533, 65536):
            table[s][i] = 3 * s + i - 65533
    lens, ask = [2**20 - 2, 2**20 - 2, 2**20 - 1, 2**20 - 1, 2**20], [1, 2, 0, 1, 0]
    for seqs in (4, 5):  # a cluster, and four kernels
        plan = ck.PagePlan(ck.PagedCache.empty(20, 1, 1, page, 4), seqs, stride)
        rc, got = plan.advance(i32(lens[:seqs]), i32(table[:seqs]), i32(ask[:seqs]), 4, window=ck.Window(*view))
        want = plain_advance(lens[:seqs], table[:seqs], ask[:seqs], 4, page, 20, view)
        assert rc == 0
        for name, a, b in zip(got._fields, got, want):
            assert a.tolist() == b, name
        assert got.status.tolist() == [0, 7, 0, 7, 3][:seqs] and got.lens.tolist()[:3] == [2**20 - 1, 2**20 - 2, 2**20 - 1]


# ---------------------------------------------------------------- sampling

@pytest.mark.parametrize("rows,vocab", [(30, 3000), (300, 700), (2, 300000)])
def test_a_table_of_zeros_gives_no_token(ck, rows, vocab):
    rng = np.random.default_rng(rows)
    logits = (rng.standard_normal((rows, vocab)) * 4 * 65536).astype(np.int64)
    logits[0, ::2] = -2**63
    zeros, t = cuda(np.zeros(4097, np.int32)), i32(rng.choice([1, 7000, 65536, 1 << 20], rows))
    for args in ({}, dict(top_k=i32([9] * rows)), dict(top_p=i32([2**23] * rows)), dict(min_p=i32([5] * rows)),
                 dict(top_k=i32([900] * rows), top_p=i32([2**24 - 1] * rows), min_p=i32([2**24] * rows))):
        rc, got = ck.sample(cuda(logits), t, cuda(np.arange(rows)), zeros, **args)
        assert rc == 0
        assert got.token.tolist() == [-1] * rows and got.prob.tolist() == [0] * rows and got.kept.tolist() == [0] * rows
    rc, got = ck.sample(cuda(logits), i32([0] * rows), cuda(np.arange(rows)), zeros)
    assert rc == 0 and got.prob.tolist() == [2**24] * rows and got.kept.tolist() == [1] * rows


@pytest.mark.parametrize("rows,vocab", [(1, 32000), (64, 32000), (200, 9000)])
def test_batches_that_all_follow_a_grammar(ck, rows, vocab):
    """Every row masked to about a third, some to one token, or none."""
    from test_gpu_streams import check_sample, settings
    rng = np.random.default_rng(rows)
    logits = (rng.standard_normal((rows, vocab)) * 3 * 65536).astype(np.int64)
    logits[rng.random((rows, vocab)) < 0.65] = -2**63
    if rows > 1:
        logits[1, :] = -2**63
        logits[2, :] = -2**63
        logits[2, vocab - 1] = 5
        logits[3, 7] = 2**40  # (one that is wider than 32 bits)
    t, k, p, m = settings(rng, rows, vocab)
    check_sample(ck, logits, t, k, p, m)
    check_sample(ck, logits, t)
