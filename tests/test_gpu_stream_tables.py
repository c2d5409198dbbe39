"""The page tables of streams with windows on the GPU, forked, packed and moved on in turn, against
plain integer forms.  All of it is integer work: tolerance 0."""
import numpy as np
import pytest

import synth
from test_gpu_paged import EXP, Setup, ck, cuda, plain_attention, pools  # noqa: F401
from test_gpu_streams import plain_advance, seen

pytestmark = pytest.mark.gpu


def i32(a):
    return cuda(np.array(a, np.int64).astype(np.uint32).view(np.int32))


def kept(n, page, view):
    """The pages of a sequence of n positions that its position n or a later one sees."""
    sinks, window = view or (0, 2**32)
    return [i for i in range(-(-n // page)) if any(t < sinks or n - t < window for t in range(i * page, (i + 1) * page))]


def plain_window_fork(lens, table, parent, grow, page, pages, view, held):
    """The fork from its definition: (table, lens, status, copies of (page, page, positions))."""
    stride, rows = len(table[0]), []
    for p, more in zip(parent, grow):
        row = {"status": 0, "mine": {}, "n": 0, "live": False}
        rows.append(row)
        if p == -1:
            continue
        if not 0 <= p < len(lens):
            row["status"] = 3
        elif lens[p] + more > min(stride * page, 2**20 - 1):
            row["status"] = 7
        else:
            mine = {i: table[p][i] for i in kept(lens[p], page, view)}
            if any(not 0 <= w < pages for w in mine.values()):
                row["status"] = 3
            else:
                row.update(live=True, mine=mine, n=lens[p], grow=more)
    live = [r for r in rows if r["live"]]
    for r in live:  # the part-filled page apart
        r["part"] = r["mine"].pop(r["n"] // page) if r["n"] % page else None
    whole = {w for r in live for w in r["mine"].values()}
    parts = [r["part"] for r in live if r["part"] is not None]
    free = [w for w in range(pages) if w not in whole and w not in parts and not held[w]]
    taken, asked, copies = set(), 0, []
    for r in live:
        part, full = r["part"], r["n"] // page
        first = part is not None and part not in taken
        taken.add(part)
        stays = first and part not in whole and not held[part] & 2
        have = full + stays
        want = -(-(r["n"] + r["grow"]) // page)
        asked += want - have
        if asked > len(free):
            r.update(status=4, mine={}, n=0)
            continue
        new = free[asked - want + have:asked]
        if stays:
            r["mine"][full] = part
        elif part is not None:
            copies.append((part, new[0], r["n"] % page))
        r["mine"].update(zip(range(have, want), new))
        r["n"] += r["grow"]
    return ([[r["mine"].get(i, -1) for i in range(stride)] for r in rows], [r["n"] for r in rows], [r["status"] for r in rows],
            copies)


def plain_window_compact(lens, table, page, pages, view):
    """Packing from its definition: (table, pages in use, status, where each page went)."""
    stride, mine, status = len(table[0]), [], []
    for n, row in zip(lens, table):
        one, rc = {}, 7 if n > min(stride * page, 2**20 - 1) else 0
        if not rc:
            one = {i: row[i] for i in kept(n, page, view)}
            if any(not 0 <= w < pages for w in one.values()):
                one, rc = {}, 3
        mine.append(one)
        status.append(rc)
    used = sorted({w for one in mine for w in one.values()})
    to = {w: w for w in used if w < len(used)}
    to.update(zip([w for w in used if w >= len(used)], [w for w in range(len(used)) if w not in to]))
    return [[to[one[i]] if i in one else -1 for i in range(stride)] for one in mine], len(used), status, to


def test_a_windowed_stream_is_forked_and_packed(ck):
    """By hand: two streams that a step has moved on, the pages behind them gone; three rows fork
    from them, then the pool is packed.  Without the window the same tables have entries outside the pool."""
    cache = ck.PagedCache.empty(16, 1, 1, 8, 4)
    plan, view = ck.PagePlan(cache, 4, 5), ck.Window(2, 4)
    rc, got = plan.advance(i32([27, 30]), i32([[0, 1, 8, 11, -1], [5, 6, 7, 9, -1]]), i32([1, 1]), 4, window=view)
    assert rc == 0 and got.table.tolist() == [[0, -1, -1, 11, -1], [5, -1, -1, 9, -1]] and got.lens.tolist() == [28, 31]
    rc, fork = plan.fork(i32([0, 0, 1]), got.lens, got.table, i32([1, 5, 2]), window=view)
    assert rc == 0 and fork.status.tolist() == [0, 0, 0] and fork.lens.tolist() == [29, 33, 33]
    assert fork.table.tolist() == [[0, -1, -1, 11, -1], [0, -1, -1, 1, 2], [5, -1, -1, 9, 3]]
    rc, packed = plan.compact(fork.lens, fork.table, window=view)
    assert rc == 0 and packed.status.tolist() == [0, 0, 0] and int(packed.used) == 7
    assert packed.table.tolist() == [[0, -1, -1, 6, -1], [0, -1, -1, 1, 2], [5, -1, -1, 4, 3]]
    rc, none = plan.fork(i32([0, 0, 1]), got.lens, got.table, i32([1, 5, 2]))
    assert rc == 0 and none.status.tolist() == [3, 3, 3]
    rc, none = plan.compact(got.lens, got.table)
    assert rc == 0 and none.status.tolist() == [3, 3]


# rows, page, stride, pages, most new positions, view, marks: in one block and over the GPU; windows that
# end inside pages, of one position, that hold everything, and none
TABLES = [
    (5, 8, 9, 60, 9, (3, 11), False),
    (1, 16, 4, 9, 20, (0, 1), False),
    (40, 8, 12, 300, 12, (9, 20), True),
    (64, 16, 40, 3000, 60, (4, 100), True),
    (30, 8, 20, 500, 20, (1000, 1), False),
    (33, 8, 20, 500, 20, None, True),
    (9, 32, 6, 40, 90, (0, 2**32 - 1), False),
    (1100, 8, 33, 20000, 30, (17, 40), True),
    (300, 8, 130, 9000, 200, (0, 64), False),
    (3, 16, 30, 66000, 100, (5, 33), True),
]


@pytest.mark.parametrize("rows,page,stride,pages,new,view,marks", TABLES)
def test_tables_forked_packed_and_moved_on_in_turn(ck, rows, page, stride, pages, new, view, marks):
    """Steps, forks and packings in turn, each against its plain form, pools included; a sequence's seen
    positions read as its ancestors wrote them."""
    rng = np.random.default_rng(rows + pages)
    k, v = pools(rng, pages, 2, 1, page, 4)
    cache = ck.PagedCache(cuda(k), cuda(v))
    plan, view = ck.PagePlan(cache, rows, stride), view and ck.Window(*view)
    lens, table, words = [0] * rows, [[-1] * stride for _ in range(rows)], [[] for _ in range(rows)]

    def check_words():
        pool = cache.k.cpu().numpy()[:, 0, 0, :, 0]
        for s in range(rows):
            for i in kept(lens[s], page, view):
                n = min(page, lens[s] - i * page)
                assert np.array_equal(pool[table[s][i], :n], words[s][i * page:i * page + n]), (s, i)

    forked = packed = 0
    for turn in range(7):
        held = np.zeros(pages, np.uint8)
        if marks:  # of pages in no table, some are others'
            apart = np.setdiff1d(np.arange(pages), [w for row in table for w in row])
            held[rng.choice(apart, len(apart) // 5, replace=False)] = rng.integers(1, 4, len(apart) // 5)
        if turn % 3 != 1:
            ask = np.where(rng.random(rows) < 0.2, 0, rng.integers(0, new + 1, rows))
            total = int(ask.sum()) + 1
            rc, got = plan.advance(i32(lens), i32(table), i32(ask), total, window=view, held=cuda(held))
            want = plain_advance(lens, table, ask.tolist(), total, page, pages, view, held)
            assert rc == 0 and [t.tolist() for t in got] == list(want)
            table, lens, starts, slots = want[:4]
            written = rng.integers(-2**31, 2**31, starts[-1]).astype(np.int32)
            cache.k.view(pages, 2, 1, page, 4)[:, 0, 0, :, 0].index_put_(
                (cuda(np.array(slots[:starts[-1]], np.int64) // page), cuda(np.array(slots[:starts[-1]], np.int64) % page)), cuda(written))
            words = [w + written[a:b].tolist() for w, a, b in zip(words, starts, starts[1:])]
        else:
            parent = rng.integers(-1, rows, rows)
            parent[rng.random(rows) < 0.5] = int(np.argmax(lens))
            grow = rng.integers(0, new + 1, rows) * (rng.random(rows) < 0.5)
            k, v = cache.k.cpu().numpy(), cache.v.cpu().numpy()
            rc, got = plan.fork(i32(parent), i32(lens), i32(table), i32(grow), held=cuda(held), window=view)
            out, out_lens, status, copies = plain_window_fork(lens, table, parent.tolist(), grow.tolist(), page, pages, view, held)
            assert rc == 0 and got.status.tolist() == status
            assert got.table.tolist() == out and got.lens.tolist() == out_lens
            for src, dst, n in copies:
                for pool in (k, v):
                    pool[dst, :, :, :n] = pool[src, :, :, :n]
            forked += status.count(0) - (parent == -1).sum()
            assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
            # (the grown positions as they are)
            pool = k[:, 0, 0, :, 0]
            words = [(words[p][:lens[p]] + [int(pool[row[t // page], t % page]) for t in range(lens[p], n)]) if n else []
                     for p, row, n in zip(parent, out, out_lens)]
            table, lens = out, out_lens
        check_words()
        k, v = cache.k.cpu().numpy(), cache.v.cpu().numpy()
        rc, got = plan.compact(i32(lens), i32(table), window=view)
        out, used, status, to = plain_window_compact(lens, table, page, pages, view)
        assert rc == 0 and got.status.tolist() == status == [0] * rows
        assert got.table.tolist() == out and int(got.used) == used
        for src, dst in to.items():
            if src != dst:
                k[dst], v[dst] = k[src], v[src]
        assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
        packed += sum(a != b for a, b in to.items())
        table = out
        check_words()
    assert forked and any(lens) and (packed or pages < 100)


def test_forks_of_windows_that_do_not_go(ck):
    """Parents outside the rows, lengths above the table, entries outside the pool inside and outside
    the window, a pool that runs out in the middle; the same for packing."""
    page, pages = 8, 20
    table = [[1, 99, 3], [4, 99, 5], [99, 6, 7], [8, 9, 10], [11, -1, -1], [-1, -1, 12]]
    lens = [25, 20, 20, 24, 4, 23]
    k, v = pools(np.random.default_rng(4), pages, 1, 1, page, 4)
    for view in (None, ck.Window(0, 3), ck.Window(1, 3), ck.Window(9, 1), ck.Window(0, 2**32 - 1)):
        for parent, grow in (([0, 1, 2, 3, 4, 5, 6, -1, 2**31], [1, 1, 1, 1, 20, 1, 1, 5, 1]), ([4, 4, 5, 5, 1], [9, 20, 0, 1, 2]),
                             ([3] * 7, [0] * 7), ([5] * 7, [0] * 7)):
            plan = ck.PagePlan(ck.PagedCache(cuda(k), cuda(v)), len(parent), 3)
            held = np.zeros(pages, np.uint8)
            held[[0, 2, 12]] = 1, 2, 2
            rc, got = plan.fork(i32(parent), i32(lens), i32(table), i32(grow), held=cuda(held), window=view)
            want = plain_window_fork(lens, table, parent, grow, page, pages, view, held)
            assert rc == 0 and [t.tolist() for t in got] == list(want[:3]), (view, parent)
        plan = ck.PagePlan(ck.PagedCache(cuda(k), cuda(v)), len(lens), 3)
        rc, got = plan.compact(i32(lens), i32(table), window=view)
        out, used, status, _ = plain_window_compact(lens, table, page, pages, view)
        assert rc == 0 and (got.table.tolist(), int(got.used), got.status.tolist()) == (out, used, status), view
    rc, _ = plan.compact(i32(lens), i32(table), window=ck.Window(3, 0))
    assert rc == 10
    rc, _ = plan.fork(i32([0]), i32(lens), i32(table), i32([0]), window=ck.Window(3, 0))
    assert rc == 10


@pytest.mark.parametrize("hd", [8, 64])
def test_attention_after_windowed_forks_and_packing(ck, hd):
    """What a windowed row sees is the same before its stream is forked and packed, and after; captured
    calls of both repeat it."""
    import torch
    page, lens, view = 16, [200, 333], ck.Window(5, 60)
    s = Setup(ck, lens, [1, 1], 4, 2, hd, page, seed=hd, spare=60)
    plan = ck.PagePlan(s.cache, 6, s.table.shape[1])
    rc, moved = plan.advance(i32(lens), i32(s.table), i32([0, 0]), 1, window=view)
    assert rc == 0 and (moved.table == -1).sum() > 12
    parent, grow = i32([1, 0, 1, 1, 0, 1]), i32([0] * 6)
    before = [t.clone() for t in (s.cache.k, s.cache.v)]
    q = s.rng.integers(-2**18, 2**18, (6, 4 * hd))
    exp, inv = cuda(EXP.view(np.int32)), synth.inv_sqrt_head(hd)
    want = np.zeros((6, 4 * hd), np.int64)
    for r, p in enumerate((1, 0, 1, 1, 0, 1)):
        t = seen(lens[p] - 1, *view)
        for h in range(4):
            K, V = (pool[s.table[p, t // page], 0, h // 2, t % page] for pool in (s.k, s.v))
            want[r, h * hd:(h + 1) * hd] = plain_attention(q[r, h * hd:(h + 1) * hd], K, V, inv)

    def serve():
        rc, fork = plan.fork(parent, moved.lens, moved.table, grow, window=view)
        assert rc == 0
        rc, packed = plan.compact(fork.lens, fork.table, window=view)
        assert rc == 0
        batch = ck.PagedBatch(packed.table, fork.lens, starts, status, 6, 1, 400)
        rc, out = ck.paged_attention(s.cache, 0, batch, queries, exp, inv, window=view)
        assert rc == 0
        return fork, packed, out

    starts, queries, status = i32(range(7)), cuda(q), torch.full((6,), -1, dtype=torch.int64, device="cuda")
    _, packed, out = serve()
    assert np.array_equal(out.cpu().numpy(), want) and packed.status.tolist() == [0] * 6
    # 333 positions: pages 0 and 17 to 20, the last part-filled; 200: pages 0 and 8 to 12
    assert int(packed.used) == 4 + 4 + 5 + 2
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fork, packed, out = serve()
    for _ in range(3):
        s.cache.k.copy_(before[0])
        s.cache.v.copy_(before[1])
        out.zero_()
        graph.replay()
        assert np.array_equal(out.cpu().numpy(), want) and fork.status.tolist() == [0] * 6
    assert status.tolist() == [-1] * 6


# ---------------------------------------------------------------- pages that two sequences would go on in

def plain_owned_advance(lens, table, new, rows, page, pages, view, held):
    """The step where a part-filled page that a sequence would go on in is named by another kept entry, or
    shared with a sequence outside the call: it asks for nothing, and its status is 10."""
    most = min(len(table[0]) * page, 2**20 - 1)
    names, refused = [], []
    for n, row in zip(lens, table):
        mine = [] if n > most else [row[i] for i in kept(n, page, view)]
        names += mine if all(0 <= w < pages for w in mine) else []
    for s, (n, row, ask) in enumerate(zip(lens, table, new)):
        if ask and n % page and n + ask <= most and all(0 <= row[i] < pages for i in kept(n, page, view)):
            last = row[n // page]
            if names.count(last) > 1 or held[last] & 2:
                refused.append(s)
    asks = [0 if s in refused else ask for s, ask in enumerate(new)]
    out, lens, starts, slots, positions, status = plain_advance(lens, table, asks, rows, page, pages, view, held)
    return out, lens, starts, slots, positions, [10 if s in refused else rc for s, rc in enumerate(status)]


def check_owned(ck, lens, table, new, rows, page, pages, view=None, held=None):
    plan = ck.PagePlan(ck.PagedCache.empty(pages, 1, 1, page, 4), len(lens), len(table[0]))
    marks = np.zeros(pages, np.uint8) if held is None else np.array(held, np.uint8)
    rc, got = plan.advance(i32(lens), i32(table), i32(new), rows, window=view, held=None if held is None else cuda(marks))
    assert rc == 0
    want = plain_owned_advance(lens, table, list(new), rows, page, pages, view, marks)
    for name, a, b in zip(got._fields, got, want):
        assert a.tolist() == b, name
    return got


def test_a_part_filled_page_of_two_sequences_is_handed_to_neither(ck):
    """By hand: slots of one page are never given to two sequences, and the others go on."""
    table = [[5, 9, -1], [3, 9, -1], [2, 4, -1], [9, 6, -1], [7, 7, -1], [8, 10, -1]]
    got = check_owned(ck, [10, 12, 11, 5, 9, 16], table, [2, 1, 1, 3, 1, 1], 9, 8, 16)
    assert got.status.tolist() == [10, 10, 0, 10, 10, 0] and got.lens.tolist() == [10, 12, 12, 5, 9, 17]
    assert got.slots.tolist() == [35, 0] + [-1] * 7 and got.table.tolist()[0] == [5, 9, -1]
    # one of the two stands still; one holds the page whole; one no longer sees it
    for lens, new, view in (([10, 12], [0, 1], None), ([16, 12], [1, 1], None), ([17, 12], [1, 1], ck.Window(0, 2))):
        got = check_owned(ck, lens, [[5, 9, 4], [3, 9, -1]], new, 9, 8, 16, view)
        assert got.status.tolist() == [0, 0 if view else 10]
    # marks: a page that is not handed out, and one that a sequence outside the call has
    for mark, status in ((1, 0), (2, 10), (3, 10)):
        held = np.zeros(16, np.uint8)
        held[[9, 5]] = mark
        got = check_owned(ck, [10, 8], [[5, 9, 4], [5, -1, -1]], [7, 1], 9, 8, 16, None, held)
        assert got.status.tolist() == [status, 0]


@pytest.mark.parametrize("seqs,stride,pages,view", [
    (3, 4, 30, None), (20, 6, 200, (3, 9)), (60, 40, 4000, None), (300, 130, 60000, (9, 500)), (2050, 20, 70000, (2, 40)),
    (40, 9, 917504, None), (40, 9, 917505, (0, 30)), (700, 800, 600000, (20, 3000))])
def test_pages_named_twice_at_random(ck, seqs, stride, pages, view):
    """Entries of other sequences in some places, whole pages and part-filled ones, in one block, in
    a cluster and over the GPU."""
    rng = np.random.default_rng(seqs + stride)
    view = view and ck.Window(*view)
    for turn in range(3):
        lens = rng.integers(0, 8 * stride - 8, seqs)
        table = rng.permutation(pages)[:seqs * stride].reshape(seqs, stride).astype(np.int64)
        for s in rng.choice(seqs, max(1, seqs // 3)):  # the last page, or any, of another
            other, i = int(rng.integers(seqs)), int(rng.integers(stride))
            table[s, lens[s] // 8 if turn != 1 else i] = table[other, lens[other] // 8 if turn else i]
        held = np.where(rng.random(pages) < 0.05, rng.integers(1, 4, pages), 0) if turn else None
        new = rng.integers(0, 4, seqs)
        got = check_owned(ck, lens.tolist(), table.tolist(), new.tolist(), 4 * seqs, 8, pages, view, held)
        if turn != 1 and seqs > 3:
            assert 10 in got.status.tolist() and 0 in got.status.tolist()


def test_what_a_fork_leaves_goes_on(ck):
    """Every row of a fork has its part-filled page to itself, also where the parent lives on outside."""
    cache = ck.PagedCache.empty(64, 1, 1, 8, 4)
    plan = ck.PagePlan(cache, 6, 6)
    table, held = [[40, 41, 42, -1, -1, -1], [50, 51, -1, -1, -1, -1]], np.zeros(64, np.uint8)
    held[[40, 41, 42]] = 3
    rc, fork = plan.fork(i32([0, 0, 1, 1, 0, 1]), i32([21, 11]), i32(table), i32([0] * 6), held=cuda(held))
    assert rc == 0 and fork.status.tolist() == [0] * 6
    rc, got = plan.advance(fork.lens, fork.table, i32([1, 2, 3, 1, 9, 1]), 32, held=cuda(held))
    assert rc == 0 and got.status.tolist() == [0] * 6
    slots = got.slots.tolist()[:17]
    assert len(set(slots)) == 17 and not {s // 8 for s in slots} & {40, 41, 42}
