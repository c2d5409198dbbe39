"""Windowed attention, the page tables' step between passes and sampling on the GPU against plain
integer implementations (the CPU oracle's steps and Python's integers), and all of them together
as a server of streams uses them.  All of it is integer work: tolerance 0."""
import numpy as np
import pytest

import oracle
import synth
from test_gpu_paged import EXP, MIN, Setup, ck, cuda, plain_attention  # noqa: F401

pytestmark = pytest.mark.gpu

ONE = 2**24


# ---------------------------------------------------------------- attention over a window

def seen(pos, sinks, window):
    t = np.arange(pos + 1)
    return t[(t < sinks) | (pos - t < window)]


class Windowed(Setup):
    """Tables without the pages that no row sees: there the entries are CK_NO_PAGE, or anything."""

    def __init__(self, ck, lens, news, heads, kv, hd, page, sinks, window, holes=(-1, 2**30), **more):
        super().__init__(ck, lens, news, heads, kv, hd, page, **more)
        self.view = ck.Window(sinks, window)
        for s, (n, length) in enumerate(zip(news, lens)):
            pages = set()
            for pos in range(max(0, length - n), length):
                pages |= set((seen(pos, sinks, window) // page).tolist())
            for i in range(self.table.shape[1]):
                if i not in pages:
                    self.table[s, i] = holes[i % len(holes)]
        self.batch.table.copy_(cuda(self.table))

    def attention(self, layer, q, inv, exp=EXP, fill=0):
        out = np.full((self.rows, self.heads * self.hd), fill, np.int64)
        for s, (n, length) in enumerate(zip(self.news, self.lens)):
            for j in range(n):
                row, pos = self.starts[s] + j, length - n + j
                t = seen(pos, *self.view)
                for h in range(self.heads):
                    kvh, c = h // (self.heads // self.kv), slice(h * self.hd, (h + 1) * self.hd)
                    out[row, c] = 0
                    if pos >= 0:
                        K, V = (pool[self.table[s, t // self.page], layer, kvh, t % self.page] for pool in (self.k, self.v))
                        out[row, c] = plain_attention(q[row, c], K, V, inv, exp)
        return out

    def run(self, ck, q, inv, layer=0, exp=EXP, **more):
        return ck.paged_attention(self.cache, layer, self.batch, cuda(q), cuda(exp.view(np.int32)), inv, window=self.view,
                                  **more)

    def queries(self, spread=65536):
        return (self.rng.standard_normal((self.rows, self.heads * self.hd)) * spread).astype(np.int64)


# lens, news, heads, kv heads, head, page, sinks, window: single tokens and chunks; windows of one, of
# odd sizes, that meet the first positions, that hold the whole sequence, that end inside pages; a
# sequence without rows and one with more rows than positions
WINDOWS = [
    ([1], [1], 1, 1, 4, 8, 0, 1),
    ([33], [1], 8, 4, 8, 16, 0, 1),
    ([33], [1], 8, 4, 8, 16, 3, 7),
    ([1, 2, 15, 16, 17, 100, 41], [1] * 7, 4, 4, 16, 16, 4, 12),
    ([257, 64, 70], [1, 1, 1], 8, 2, 64, 32, 4, 64),
    ([300], [1], 3, 3, 128, 256, 9, 20),
    ([1025], [1], 32, 32, 64, 64, 4, 512),
    ([5000], [1], 4, 1, 128, 16, 8, 2048),
    ([9001, 40], [1, 1], 4, 1, 64, 32, 4, 4097),
    ([0, 5, 9], [1, 0, 2], 2, 2, 32, 8, 1, 3),
    ([3], [5], 2, 1, 8, 8, 0, 2),
    ([130, 67], [130, 3], 4, 2, 64, 16, 4, 33),
    ([200], [200], 2, 2, 128, 32, 0, 40),
    ([77, 300, 12], [20, 129, 12], 4, 4, 32, 64, 70, 5),
    ([513], [65], 8, 1, 64, 64, 17, 100),
    ([700], [40], 6, 2, 16, 8, 2, 300),
    ([260], [129], 2, 2, 4, 16, 0, 9),
    ([900], [2], 4, 2, 64, 16, 5, 128),
    ([900], [3], 4, 4, 32, 8, 24, 257),
    ([50, 60], [1, 1], 4, 4, 64, 16, 100, 8),
    ([50, 60], [1, 1], 4, 4, 64, 16, 4, 2**32 - 1),
    ([901], [300], 32, 8, 128, 128, 0, 1),
]
# work enough for the tensor-core tiles
WINDOW_TILES = [
    ([1900, 733], [70, 129], 32, 8, 64, 16, 4, 500),
    ([1640], [200], 16, 16, 128, 32, 0, 333),
    ([2030, 40], [129, 40], 8, 1, 64, 8, 13, 700),
    ([2100], [20], 32, 4, 128, 64, 64, 1001),
    ([1077, 530], [90, 2], 48, 3, 64, 32, 1, 256),
    ([300, 1500, 5], [0, 65, 5], 32, 32, 64, 256, 300, 511),
    ([640], [640], 16, 4, 64, 64, 4, 64),
]


@pytest.mark.parametrize("lens,news,heads,kv,hd,page,sinks,window", WINDOWS + WINDOW_TILES)
def test_window_against_the_plain_form(ck, lens, news, heads, kv, hd, page, sinks, window):
    s = Windowed(ck, lens, news, heads, kv, hd, page, sinks, window, seed=hd + len(lens))
    tiles = ck.paged_attention_work(s.cache, s.batch, heads, window=s.view).numel() > 1 << 20
    assert tiles == ((lens, news, heads, kv, hd, page, sinks, window) in WINDOW_TILES)
    q, inv = s.queries(), synth.inv_sqrt_head(hd)
    for layer in (0, 1):
        rc, out = s.run(ck, q, inv, layer)
        assert rc == 0
        assert np.array_equal(out.cpu().numpy(), s.attention(layer, q, inv))
    assert s.batch.errors() == [None] * len(lens)


@pytest.mark.parametrize("lens,news,heads,kv,hd,page,sinks,window", WINDOW_TILES)
def test_windowed_tiles_give_the_same_bits_every_time(ck, lens, news, heads, kv, hd, page, sinks, window):
    import torch
    s = Windowed(ck, lens, news, heads, kv, hd, page, sinks, window, seed=5)
    q, exp = cuda(s.queries()), cuda(EXP.view(np.int32))
    rc, first = ck.paged_attention(s.cache, 0, s.batch, q, exp, 1 << 21, window=s.view)
    assert rc == 0
    for _ in range(100):
        rc, out = ck.paged_attention(s.cache, 0, s.batch, q, exp, 1 << 21, window=s.view)
        assert rc == 0 and torch.equal(out, first)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("q_spread,kv_spread", [(2**62, 65536), (65536, 2**31 - 1), (2**31, 2**31 - 1),
                                                (2**23 + 5, 2**23 + 5), (1, 1), (0, 65536)])
def test_window_over_the_whole_range_of_values(ck, new, q_spread, kv_spread):
    heads, kv = (4, 2) if new == 1 else (32, 4)
    s = Windowed(ck, [900], [new], heads, kv, 64, 16, 4, 450, seed=1)
    s.k[:] = s.rng.integers(-kv_spread - 1, kv_spread + 1, s.k.shape)
    s.v[:] = s.rng.integers(-kv_spread - 1, kv_spread + 1, s.v.shape)
    s.cache.k.copy_(cuda(s.k))
    s.cache.v.copy_(cuda(s.v))
    q = s.rng.integers(-q_spread, q_spread + 1, (s.rows, heads * 64))
    inv = synth.inv_sqrt_head(64)
    rc, out = s.run(ck, q, inv, 1)
    assert rc == 0
    assert np.array_equal(out.cpu().numpy(), s.attention(1, q, inv))


@pytest.mark.parametrize("lens,news,heads,kv,hd", [([700, 650], [1, 1], 4, 4, 64), ([1200, 900], [60, 70], 32, 8, 64),
                                                   ([1200, 900], [60, 70], 16, 4, 128), ([300, 290], [5, 9], 2, 1, 16)])
def test_positions_outside_the_window_count_for_nothing(ck, lens, news, heads, kv, hd):
    """The words next to the window and to the first positions would win every softmax, and their
    values are the largest there are: none is seen."""
    s = Windowed(ck, lens, news, heads, kv, hd, 16, 5, 203, seed=9)
    q, inv = np.abs(s.queries()) + 1, synth.inv_sqrt_head(hd)
    for i, (n, length) in enumerate(zip(news, lens)):
        pos = range(length - n, length)
        any_row = set().union(*(seen(p, *s.view).tolist() for p in pos))
        for t in range(length):
            page = s.table[i, t // 16]
            if t not in any_row and 0 <= page < s.pages:
                s.k[page, :, :, t % 16] = 127 * 65793
                s.v[page, :, :, t % 16] = 127 * 65793
    s.cache.k.copy_(cuda(s.k))
    s.cache.v.copy_(cuda(s.v))
    rc, out = s.run(ck, q, inv)
    assert rc == 0
    assert np.array_equal(out.cpu().numpy(), s.attention(0, q, inv))


@pytest.mark.parametrize("lens,news,heads,kv,hd,page,sinks,window",
                         [WINDOWS[6], WINDOWS[11], WINDOWS[13], WINDOW_TILES[0], WINDOW_TILES[1]])
def test_a_window_that_holds_everything_is_the_whole_cache(ck, lens, news, heads, kv, hd, page, sinks, window):
    import torch
    s = Setup(ck, lens, news, heads, kv, hd, page, seed=2)
    q, exp = cuda((s.rng.standard_normal((s.rows, heads * hd)) * 65536).astype(np.int64)), cuda(EXP.view(np.int32))
    rc, want = ck.paged_attention(s.cache, 0, s.batch, q, exp, 1 << 21)
    assert rc == 0
    longest = max(lens)
    for view in (ck.Window(0, longest), ck.Window(longest, 1), ck.Window(2**32 - 1, 2**32 - 1), ck.Window(longest - 1, 1),
                 ck.Window(0, longest - 1), ck.Window(longest // 2, longest // 2 + 1)):
        rc, out = ck.paged_attention(s.cache, 0, s.batch, q, exp, 1 << 21, window=view)
        assert rc == 0
        if view != ck.Window(0, longest - 1):  # (the last row of the longest sequence misses its first position)
            assert torch.equal(out, want)
    assert not torch.equal(out, torch.zeros_like(out))


def test_window_bounds_above_the_lengths(ck):
    """Launch bounds far above what the arrays say, rows of no sequence before and behind, strided
    queries: what no row owns stays as it was."""
    import torch
    for news, heads, kv, hd in (([1, 1], 4, 2, 64), ([60, 33], 32, 8, 64), ([4, 2], 2, 2, 16)):
        s = Windowed(ck, [800, 420], news, heads, kv, hd, 16, 4, 90, seed=hd, lead=3, tail=5)
        table = cuda(np.concatenate([s.table, np.full((2, 5000 // 16), -1, np.int32)], 1))
        s.batch = ck.PagedBatch(table, cuda(np.array(s.lens, np.int32)), cuda(s.starts), None, s.rows, s.rows, 5000)
        wide = (s.rng.standard_normal((s.rows, heads * hd + 6)) * 65536).astype(np.int64)
        out = torch.full((s.rows, heads * hd), 7, dtype=torch.int64, device="cuda")
        rc, _ = ck.paged_attention(s.cache, 1, s.batch, cuda(wide)[:, 2:2 + heads * hd], cuda(EXP.view(np.int32)), 1 << 21,
                                   out=out, window=s.view)
        assert rc == 0 and s.batch.errors() == [None, None]
        assert np.array_equal(out.cpu().numpy(), s.attention(1, wide[:, 2:], 1 << 21, fill=7))


@pytest.mark.parametrize("news,heads,kv,hd", [([1, 1, 1], 4, 2, 64), ([40, 40, 40], 32, 4, 64), ([3, 5, 2], 2, 1, 8)])
def test_bad_pages_in_and_outside_of_the_window(ck, news, heads, kv, hd):
    """A page outside the pool counts as zeros and is reported where a row sees it, and only there; a
    sequence longer than the bound is skipped."""
    import torch
    s = Windowed(ck, [700, 703, 2000], news, heads, kv, hd, 16, 4, 100, seed=3, holes=(-1,))
    bad = 690 // 16
    s.table[0, bad] = s.pages + 3
    first_seen = min(i for i in range(1, 44) if s.table[1, i] >= 0)
    s.table[1, first_seen - 1] = 2**30         # not seen
    batch = ck.PagedBatch(cuda(s.table), cuda(np.array(s.lens, np.int32)), cuda(s.starts), None, s.rows, max(news), 1000)
    q = s.queries()
    out = torch.full((s.rows, heads * hd), 7, dtype=torch.int64, device="cuda")
    rc, _ = ck.paged_attention(s.cache, 0, batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 21, out=out, window=s.view)
    assert rc == 0
    assert batch.errors() == [(bad * 16, 0, ck.BAD_PAGE, 0), None, (0, 0, ck.BAD_SEQUENCE, 0)]
    s.k, s.v = (np.concatenate([p, np.zeros_like(p[:1])]) for p in (s.k, s.v))
    s.table[0, bad] = s.pages                   # a page of zeros
    want = s.attention(0, q, 1 << 21, fill=7)
    skipped = s.starts[2]
    assert np.array_equal(out.cpu().numpy()[:skipped], want[:skipped])
    assert (out[skipped:] == 7).all()


def test_windows_on_two_streams_and_captured(ck):
    import torch
    jobs = []
    for new in (1, 60):
        s = Windowed(ck, [1500, 920], [new, new], 32, 4, 64, 16, 4, 400, seed=new)
        q = [s.queries() for _ in range(2)]
        jobs.append((s, q, [s.attention(0, x, 1 << 21) for x in q]))
    exp = cuda(EXP.view(np.int32))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = [[cuda(x) for x in q] for _, q, _ in jobs]
    torch.cuda.synchronize()
    outs = []
    for turn in range(20):
        for (s, _, _), d, stream in zip(jobs, dev, streams):
            outs.append(ck.paged_attention(s.cache, 0, s.batch, d[turn % 2], exp, 1 << 21, stream=stream, window=s.view))
    torch.cuda.synchronize()
    for i, (rc, out) in enumerate(outs):
        assert rc == 0 and np.array_equal(out.cpu().numpy(), jobs[i % 2][2][i // 2 % 2])
    for (s, q, want), d in zip(jobs, dev):
        place, out = d[0].clone(), torch.zeros_like(d[0])
        work = ck.paged_attention_work(s.cache, s.batch, 32, window=s.view)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rc, _ = ck.paged_attention(s.cache, 0, s.batch, place, exp, 1 << 21, out=out, work=work, window=s.view)
        assert rc == 0
        for turn in (1, 0, 1):
            place.copy_(d[turn])
            out.zero_()
            graph.replay()
            assert np.array_equal(out.cpu().numpy(), want[turn])


def test_window_scratch_too_small_is_refused(ck):
    s = Windowed(ck, [1900, 733], [70, 129], 32, 8, 64, 16, 4, 500)
    n = ck.paged_attention_work(s.cache, s.batch, 32, window=s.view).numel()
    import torch
    work = torch.empty(n - 256 if n > 256 else 0, dtype=torch.uint8, device="cuda")
    rc, _ = s.run(ck, s.queries(), 1 << 21, work=torch.empty(256, dtype=torch.uint8, device="cuda")[:0] if n <= 256 else work)
    assert rc in (4, 10)  # (10: an empty buffer has no address)
    rc, _ = ck.paged_attention(s.cache, 0, s.batch, cuda(s.queries()), cuda(EXP.view(np.int32)), 1 << 21,
                               window=ck.Window(4, 0), work=work)
    assert rc == 10


def test_windows_and_steps_beyond_32_bits_of_words(ck):
    """Pages at the far end of pools of over 2^32 words each: a step hands them out, its slots are
    stored to, windows read them (chunks, chunks of large queries, single tokens)."""
    import torch
    page, hd, pages, n = 256, 128, 131072 + 64, 300
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 36 GB of device memory")
    cache = ck.PagedCache.empty(pages, 1, 1, page, hd)
    rng = np.random.default_rng(9)
    top, view, inv, exp = pages - 1, ck.Window(3, 40), synth.inv_sqrt_head(hd), cuda(EXP.view(np.int32))
    held = torch.ones(pages, dtype=torch.uint8, device="cuda")
    held[[top - 40, top]] = 0
    plan = ck.PagePlan(cache, 1, 4)
    rc, step = plan.advance(cuda(np.zeros(1, np.int32)), cuda(np.full((1, 4), -1, np.int32)), cuda(np.array([n], np.int32)), n,
                            window=view, held=held)
    assert rc == 0 and step.status.tolist() == [0] and step.table.tolist() == [[top - 40, top, -1, -1]]
    slots = np.concatenate([(top - 40) * page + np.arange(page), top * page + np.arange(n - page)])
    assert np.array_equal(step.slots.cpu().numpy(), slots)
    k, v = ((rng.standard_normal((n, hd)) * 65536).astype(np.int64) for _ in range(2))
    for pool, words in ((cache.k, k), (cache.v, v)):
        pool.view(-1, hd)[step.slots] = cuda(words.astype(np.int32))
    for spread, new in ((65536, n), (2**40, n), (65536, 1)):
        q = (rng.standard_normal((new, 32 * hd)) * spread).astype(np.int64)
        batch = ck.PagedBatch(step.table, step.lens, cuda(np.array([0, new], np.int32)), None, new, new, n)
        assert (ck.paged_attention_work(cache, batch, 32, window=view).numel() > 1 << 20) == (new > 1)  # the tiles
        rc, out = ck.paged_attention(cache, 0, batch, cuda(q), exp, inv, window=view)
        assert rc == 0 and batch.errors() == [None]
        for row in {0, 130, 299} if new > 1 else (0,):
            t = seen(n - new + row, *view)
            for h in (0, 17, 31):
                c = slice(h * hd, (h + 1) * hd)
                assert np.array_equal(out[row, c].cpu().numpy(), plain_attention(q[row, c], k[t], v[t], inv))


# ---------------------------------------------------------------- the tables between passes

def plain_advance(lens, table, new, rows, page, pages, view=None, held=()):
    """The step from its definition, one sequence after the other."""
    stride = len(table[0])
    most = min(stride * page, 2**20 - 1)
    out, used = [], {p for p in range(pages) if len(held) and held[p]}
    for n, row, ask in zip(lens, table, new):
        sinks, window = view or (0, 2**32 - 1)
        mine = {i: row[i] for i in range(min(-(-n // page), stride)) if i * page < sinks or n - ((i + 1) * page - 1) < window}
        status = 3 if n > most or any(not 0 <= p < pages for p in mine.values()) else 7 if n + ask > most else 0
        if status == 3:
            mine, n = {}, 0
        used |= set(mine.values())
        out.append([mine, n, ask, status])
    free = [p for p in range(pages) if p not in used]
    pages_asked = rows_asked = 0
    starts, slots, positions = [0], [], []
    for seq in out:
        mine, n, ask, status = seq
        granted = 0
        if status == 0:
            have, want = -(-n // page), -(-(n + ask) // page)
            pages_asked, rows_asked = pages_asked + want - have, rows_asked + ask
            if (want > have and pages_asked > len(free)) or (ask and rows_asked > rows):
                seq[3] = 4
            else:
                mine.update(zip(range(have, want), free[pages_asked - want + have:]))
                seq[1], granted = n + ask, ask
                positions += range(n, n + ask)
                slots += [mine[t // page] * page + t % page for t in range(n, n + ask)]
        starts.append(starts[-1] + granted)
    rest = [-1] * (rows - starts[-1])
    return ([[seq[0].get(i, -1) for i in range(stride)] for seq in out], [seq[1] for seq in out], starts, slots + rest,
            positions + rest, [seq[3] for seq in out])


def check_advance(ck, lens, table, new, rows, page, pages, view=None, held=None, layers=1):
    plan = ck.PagePlan(ck.PagedCache.empty(pages, layers, 1, page, 4), len(lens), len(table[0]))
    i32 = lambda a: cuda(np.array(a, np.int64).astype(np.uint32).view(np.int32))
    rc, got = plan.advance(i32(lens), i32(table), i32(new), rows, window=view,
                           held=None if held is None else cuda(np.array(held, np.uint8)))
    assert rc == 0
    want = plain_advance(lens, table, new, rows, page, pages, view, [] if held is None else held)
    for name, a, b in zip(got._fields, got, want):
        assert a.tolist() == b, name
    return got


def test_advance_gives_back_grows_and_places(ck):
    """Five sequences, by hand: one grows in its page, one gets a page, one takes a chunk, one stands
    still behind its window, one begins."""
    table = [[5, 9, -1, -1, -1], [2, 3, -1, -1, -1], [7, -1, -1, -1, -1], [0, 1, 8, 11, -1], [-1] * 5]
    got = check_advance(ck, [10, 16, 3, 27, 0], table, [1, 1, 14, 0, 2], 20, 8, 16, ck.Window(2, 4))
    assert got.table.tolist() == [[5, 9, -1, -1, -1], [2, 3, 1, -1, -1], [7, 4, 6, -1, -1], [0, -1, -1, 11, -1],
                                  [8, -1, -1, -1, -1]]
    assert got.lens.tolist() == [11, 17, 17, 27, 2] and got.starts.tolist() == [0, 1, 2, 16, 16, 18]
    assert got.slots.tolist()[:4] == [74, 8, 59, 60] and got.positions.tolist()[-4:] == [0, 1, -1, -1]


def test_advance_of_what_does_not_go(ck):
    """Lengths above the table and above 2^20 - 1, entries outside the pool inside and outside the
    window, tables that are full, requests beyond the pages and the rows: each is its own, and the
    sequences behind it that need nothing go on."""
    table = [[1, 2, 3], [4, 99, 5], [99, 6, 7], [8, 9, 10], [11, -1, -1], [12, -1, -1], [13, 14, -1], [15, -1, -1]]
    lens, new = [25, 20, 20, 24, 4, 5, 9, 0], [1, 1, 1, 1, 20, 1, 1, 0]
    got = check_advance(ck, lens, table, new, 6, 8, 17, ck.Window(0, 3))
    assert got.status.tolist() == [3, 0, 0, 7, 4, 4, 4, 0]
    got = check_advance(ck, lens, table, new, 60, 8, 17, ck.Window(0, 3))
    assert got.status.tolist() == [3, 0, 0, 7, 0, 0, 0, 0]
    got = check_advance(ck, lens, table, new, 60, 8, 17, ck.Window(1, 3))
    assert got.status.tolist() == [3, 0, 3, 7, 0, 0, 0, 0]
    got = check_advance(ck, lens, table, new, 60, 8, 17, None)
    assert got.status.tolist()[1] == 3
    got = check_advance(ck, lens, table, new, 60, 8, 17, ck.Window(0, 3), held=[1] * 17)
    assert got.status.tolist() == [3, 0, 0, 7, 4, 0, 0, 0]
    huge = [2**32 - 1, 2**31, 2**20 - 1, 0, 5, 1, 8, 2**20]
    check_advance(ck, huge, table, [2**32 - 1] * 8, 5, 8, 17, ck.Window(0, 3))
    check_advance(ck, [0] * 8, table, [2**32 - 1, 1, 2**20, 2**31, 9, 1, 1, 24], 2**20, 8, 17, None)


@pytest.mark.parametrize("seqs,page,stride,pages,rows,new,view,held", [
    (1, 8, 1, 1, 1, 1, None, False), (1, 256, 3, 5, 300, 250, None, False), (3, 16, 40, 200, 9, 3, (4, 37), True),
    (33, 8, 70, 900, 100, 5, (0, 1), False), (64, 16, 513, 5000, 64, 1, (4, 1000), True),
    (200, 16, 33, 3000, 2**20, 90, (70, 100), True), (1025, 32, 20, 40000, 3000, 4, None, False),
    (2500, 8, 64, 70001, 5000, 3, (9, 200), True), (5000, 64, 3, 65537, 5000, 1, None, True),
    # long tables: pages at their beginnings and in windows far behind, and all of them
    (20, 8, 700, 30000, 2**20, 5, (20, 1500), True), (40, 16, 513, 30000, 2**20, 1, (4, 1024), False),
    (9, 8, 1100, 12000, 2**20, 2, None, False), (70, 8, 300, 20000, 2**20, 9, (1200, 3), True),
    # tables too large for one cluster
    (1500, 8, 400, 400000, 2**20, 5, (20, 700), True), (600, 16, 1000, 250000, 2**20, 1, None, False)])
def test_advance_step_after_step(ck, seqs, page, stride, pages, rows, new, view, held):
    """Several steps from empty tables, whatever is granted, against the plain form."""
    rng = np.random.default_rng(seqs + pages)
    plan = ck.PagePlan(ck.PagedCache.empty(pages, 1, 1, page, 4), seqs, stride)
    mask = rng.random(pages) < 0.3 if held else None
    view = view and ck.Window(*view)
    lens, table = [0] * seqs, [[-1] * stride for _ in range(seqs)]
    lens_d, table_d = cuda(np.array(lens, np.int32)), cuda(np.array(table, np.int32))
    for step in range(6):
        ask = np.where(rng.random(seqs) < 0.2, 0, rng.integers(0, (new if step % 2 else stride * page // 3) + 1, seqs))
        rc, got = plan.advance(lens_d, table_d, cuda(ask.astype(np.int32)), rows, window=view,
                               held=None if mask is None else cuda(mask.astype(np.uint8)))
        assert rc == 0
        want = plain_advance(lens, table, ask.tolist(), rows, page, pages, view, [] if mask is None else mask)
        for name, a, b in zip(got._fields, got, want):
            assert a.tolist() == b, (name, step)
        table, lens = want[0], want[1]
        table_d, lens_d = got.table, got.lens
    assert any(lens)


def test_advance_keeps_pages_that_sequences_share(ck):
    """A page that one sequence gives back and another still keeps is not handed out."""
    table = [[3, 4, 5, -1], [3, 4, 6, -1]]
    got = check_advance(ck, [20, 17], table, [5, 7], 20, 8, 8, ck.Window(0, 5))
    assert got.table.tolist() == [[-1, -1, 5, 0], [-1, 4, 6, -1]]


def test_advance_of_a_pool_past_2_20_pages(ck):
    """Few sequences and more pages than one cluster keeps apart."""
    pages = 2**20 + 77
    held = np.ones(pages, np.uint8)
    held[[5, 9, 2**20 - 1, 2**20, 2**20 + 76]] = 0
    table = [[2**20 + 70, 2**20 + 75, -1, -1], [2**20 + 76, -1, -1, -1]]
    got = check_advance(ck, [16, 3], table, [10, 6], 20, 8, pages, None, held)
    assert got.table.tolist() == [[2**20 + 70, 2**20 + 75, 5, 9], [2**20 + 76, 2**20 - 1, -1, -1]]
    check_advance(ck, [16, 3], table, [17, 6], 20, 8, pages, ck.Window(0, 2), held)


def test_advance_on_two_streams_at_once(ck):
    """Two plans of one pool's shape, small tables and ones past a cluster, each on its stream."""
    import torch
    rng = np.random.default_rng(8)
    for seqs, stride, pages in ((30, 20, 500), (1500, 400, 300000)):
        cache = ck.PagedCache.empty(pages, 1, 1, 8, 4)
        plans, streams = [ck.PagePlan(cache, seqs, stride) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
        state, want, outs = [], [], []
        for _ in range(2):
            new = rng.integers(0, 90, seqs)
            state.append((cuda(np.zeros(seqs, np.int32)), cuda(np.full((seqs, stride), -1, np.int32)),
                          cuda(new.astype(np.int32))))
            want.append(plain_advance([0] * seqs, [[-1] * stride] * seqs, new.tolist(), 2**17, 8, pages, (3, 20)))
        torch.cuda.synchronize()
        for turn in range(12):
            i = turn % 2
            outs.append(plans[i].advance(*state[i], 2**17, window=ck.Window(3, 20), stream=streams[i]))
        torch.cuda.synchronize()
        for turn, (rc, got) in enumerate(outs):
            assert rc == 0 and [x.tolist() for x in got] == list(want[turn % 2])


def test_advance_captured_on_another_stream_and_refusals(ck):
    import torch
    cache = ck.PagedCache.empty(40, 1, 1, 8, 4)
    plan, side = ck.PagePlan(cache, 4, 6), torch.cuda.Stream()
    lens, table = cuda(np.zeros(4, np.int32)), cuda(np.full((4, 6), -1, np.int32))
    new = cuda(np.array([3, 9, 0, 17], np.int32))
    side.wait_stream(torch.cuda.current_stream())
    rc, got = plan.advance(lens, table, new, 32, window=ck.Window(1, 5), stream=side)
    side.synchronize()
    assert rc == 0
    want = plain_advance([0] * 4, table.tolist(), new.tolist(), 32, 8, 40, (1, 5))
    assert [t.tolist() for t in got] == list(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # a step that feeds itself
        rc, got = plan.advance(lens, table, new, 32, window=ck.Window(1, 5))
        lens.copy_(got.lens)
        table.copy_(got.table)
    assert rc == 0
    l, t = [0] * 4, [[-1] * 6 for _ in range(4)]
    for _ in range(3):
        want = plain_advance(l, t, new.tolist(), 32, 8, 40, (1, 5))
        graph.replay()
        assert [x.tolist() for x in got] == list(want)
        t, l = want[0], want[1]
    for bad in (dict(rows=0), dict(rows=2**20 + 1), dict(new=new[:3]), dict(new=new.long()), dict(lens=lens[:2]),
                dict(table=table[:, :5]), dict(held=cuda(np.zeros(39, np.uint8)))):
        args = dict(lens=lens, table=table, new=new, rows=32)
        args.update(bad)
        with pytest.raises(ValueError):
            plan.advance(**args)
    with pytest.raises(ValueError, match="room"):
        plan.advance(cuda(np.zeros(5, np.int32)), cuda(np.full((5, 6), -1, np.int32)), cuda(np.zeros(5, np.int32)), 8)
    assert plan.advance(lens, table, new, 32, window=ck.Window(4, 0))[0] == 10


# ---------------------------------------------------------------- sampling

def plain_sample(logits, t, k, p, m, random, exp=EXP):
    """One row from the definition, in Python's integers: (token, probability, kept)."""
    allowed = [i for i, l in enumerate(logits.tolist()) if l != MIN]
    if not allowed or t > 16 << 16:
        return -1, 0, 0
    values = logits.tolist()
    top = max(values[i] for i in allowed)
    order = sorted(allowed, key=lambda i: (top - values[i], i))
    if t == 0:
        return order[0], ONE, 1
    d = {i: top - values[i] for i in order}
    e = {i: int(exp[4096 if d[i] >= 16 * t else 256 * d[i] // t]) for i in order}
    n = min(k, len(order)) if k else len(order)
    if p < ONE:
        target, total = sum(e[i] for i in order[:n]) * p >> 24, 0
        for count, i in enumerate(order[:n], 1):
            total += e[i]
            if total >= target:
                n = count
                break
    if m:
        n = max(1, min(n, sum(e[i] << 24 >= min(m, ONE) * int(exp[0]) for i in order)))
    keep = sorted(order[:n])
    weight = sum(e[i] for i in keep)
    draw = random % weight
    for i in keep:
        if draw < e[i]:
            return i, (e[i] << 24) // weight, n
        draw -= e[i]


def check_sample(ck, logits, t, k=None, p=None, m=None, random=None, exp=EXP, seed=0):
    rows = len(logits)
    rng = np.random.default_rng(seed)
    if random is None:
        random = rng.integers(0, 2**64, rows, dtype=np.uint64)
    u32 = lambda a: None if a is None else cuda(np.array(a, np.uint32).view(np.int32))
    rc, got = ck.sample(cuda(logits) if isinstance(logits, np.ndarray) else logits, u32(t), cuda(random.view(np.int64)),
                        cuda(exp.view(np.int32)), top_k=u32(k), top_p=u32(p), min_p=u32(m))
    assert rc == 0
    host = logits if isinstance(logits, np.ndarray) else logits.cpu().numpy()
    each = lambda a, off: [off] * rows if a is None else [int(x) for x in a]
    want = [plain_sample(*x, exp) for x in zip(host, each(t, 0), each(k, 0), each(p, ONE), each(m, 0), random.tolist())]
    assert list(zip(*(x.tolist() for x in got))) == want
    return got


def settings(rng, rows, vocab):
    t = np.where(rng.random(rows) < 0.1, 0, rng.choice([1, 7000, 30000, 65536, 98304, 16 << 16], rows))
    k = np.where(rng.random(rows) < 0.3, 0, rng.integers(1, max(2, min(vocab + 3, 300)), rows))
    p = np.where(rng.random(rows) < 0.3, ONE, rng.integers(0, ONE + 2, rows))
    m = np.where(rng.random(rows) < 0.3, 0, (rng.random(rows) ** 4 * (ONE + 2)).astype(np.int64))
    return t, k, p, m


@pytest.mark.parametrize("rows,vocab", [(1, 1), (5, 2), (40, 7), (33, 31), (20, 33), (64, 512), (9, 4095), (9, 4096), (9, 4097),
                                        (17, 32000), (6, 32768), (6, 32769), (3, 65537), (2, 200000)])
@pytest.mark.parametrize("spread", [0.5, 3.0])
def test_sampling_against_the_plain_form(ck, rows, vocab, spread):
    rng = np.random.default_rng(rows + vocab)
    logits = (rng.standard_normal((rows, vocab)) * spread * 65536).astype(np.int64)
    t, k, p, m = settings(rng, rows, vocab)
    check_sample(ck, logits, t, k, p, m)
    check_sample(ck, logits, t)
    check_sample(ck, logits, t, k)
    check_sample(ck, logits, t, None, p)
    check_sample(ck, logits, t, None, None, m)
    logits[rng.random((rows, vocab)) < 0.7] = MIN
    check_sample(ck, logits, t, k, p, m)


@pytest.mark.parametrize("rows,vocab", [(4, 262143), (4, 262144), (4, 262145), (3, 300001), (1, 2**20)])
def test_sampling_of_vocabularies_past_a_clusters_memory(ck, rows, vocab):
    """Rows whose words fit the shared memory of a cluster and the ones behind: drawn ones, ones of
    ties, distances past 32 bits, masks, with filters and without."""
    rng = np.random.default_rng(vocab)
    logits = (rng.standard_normal((rows, vocab)) * 2 * 65536).astype(np.int64)
    logits[-1, 1::2] = MIN
    t = [65536, 30000, 1 << 20, 65536][:rows]
    check_sample(ck, logits, t, [0, 900, 7, vocab // 3][:rows], [ONE // 2, ONE, ONE - 1, ONE][:rows], [0, 9000, 0, 0][:rows])
    check_sample(ck, logits, t)
    if rows > 1:
        logits[0] = 77
        logits[1] = rng.integers(-2**62, 2**62, vocab)
        logits[2] >>= 14
        check_sample(ck, logits, [0] + t[1:], [3, vocab // 5, vocab // 2, 5][:rows], [ONE, ONE, ONE - 1, ONE][:rows])
        check_sample(ck, logits, t, [vocab - 1] * rows)


@pytest.mark.parametrize("vocab", [3, 512, 40000, 300000])
def test_sampling_keeps_everything_where_filters_ask_for_more(ck, vocab):
    """A top-k of the vocabulary and above, a top-p of one and above, a min-p of nothing: the rows
    without filters."""
    import torch
    rng = np.random.default_rng(vocab)
    logits = cuda((rng.standard_normal((6, vocab)) * 65536).astype(np.int64))
    i32 = lambda *a: cuda(np.array(a, np.uint32).view(np.int32))
    random, exp, t = cuda(rng.integers(-2**63, 2**63, 6)), cuda(EXP.view(np.int32)), i32(*[65536] * 6)
    rc, want = ck.sample(logits, t, random, exp)
    assert rc == 0 and want.kept.tolist() == [vocab] * 6
    rc, got = ck.sample(logits, t, random, exp, top_k=i32(vocab, vocab + 1, 2**32 - 1, 0, vocab, 2**31),
                        top_p=i32(ONE, ONE + 1, 2**32 - 1, 2**31, ONE, ONE), min_p=i32(*[0] * 6))
    assert rc == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_oracle_samples_the_same(ck):
    """Without filters and with the generator's outputs: the oracle's token and its probability."""
    rng = np.random.default_rng(1)
    logits = (rng.standard_normal((60, 700)) * 2 * 65536).astype(np.int64)
    t = rng.integers(1, 1 << 18, 60)
    random, want, state = [], [], 99
    for row, temp in zip(logits, t):
        one = oracle.sample(row, int(temp), EXP, state)
        state, x = oracle.xorshift_next(state)
        assert one["draw"] == x % one["sum"]
        random.append(x)
        want.append(one["token"])
    got = check_sample(ck, logits, t, random=np.array(random, np.uint64))
    assert got.token.tolist() == want


@pytest.mark.parametrize("vocab", [300, 5000, 40000])
def test_sampling_of_ties(ck, vocab):
    """Equal logits, and a few values: the kept tokens end among equals, more than are ranked by
    counting, and the lowest tokens stay."""
    rng = np.random.default_rng(vocab)
    logits = np.stack([np.zeros(vocab, np.int64), np.full(vocab, 2**62), np.full(vocab, MIN + 1),
                       rng.integers(0, 2, vocab) << 16, rng.integers(0, 3, vocab) << 14, rng.integers(0, 2, vocab)])
    rows = len(logits)
    for k in (1, 2, 257, vocab // 2, vocab - 1):
        check_sample(ck, logits, [65536] * rows, [k] * rows, seed=k)
        check_sample(ck, logits, [16 << 16] * rows, [k] * rows, [ONE // 3] * rows, seed=k)
    check_sample(ck, logits, [0] * rows)
    check_sample(ck, logits, [20000] * rows, None, [1, ONE // 7, ONE // 2, ONE - 1, 0, 2], [0, 1, 1000, ONE, ONE + 9, 2**32 - 1])


@pytest.mark.parametrize("vocab", [2000, 33000])
def test_sampling_in_the_tail_of_the_table(ck, vocab):
    """Top-k ends among tokens sixteen temperatures and more away, next to one another, far apart, and
    with distances past 32 bits up to nearly 2^64."""
    rng = np.random.default_rng(vocab)
    spans = [2**20, 2**33, 2**50, 2**63 - 1, 2**63 - 1]
    logits = np.stack([rng.integers(-s, 0, vocab) for s in spans] + [-(2**40) - rng.integers(0, 500, vocab),
                                                                     rng.integers(0, 2, vocab) - 2**45])
    logits[:, vocab // 3] = 1000
    logits[4, vocab // 3] = 2**63 - 1
    logits[4, :20] = MIN + 1 + np.arange(20)[::-1] // 2
    rows = len(logits)
    for t in (1, 300, 40000):
        for k in (1, 2, 3, 100, 700, vocab - 11, vocab - 1):
            check_sample(ck, logits, [t] * rows, [k] * rows, seed=k)
            check_sample(ck, logits, [t] * rows, [k] * rows, [ONE - 1] * rows, seed=k)


def test_sampling_of_masked_rows_and_odd_settings(ck):
    """Rows whose mask leaves one token or nothing, temperatures above the limit, settings at the
    ends of 32 bits, draws at both ends of the weights."""
    logits = np.full((8, 900), MIN, np.int64)
    logits[1, 899] = -2**63 + 1
    logits[2, 5] = 2**63 - 1
    logits[3, 700:] = 12
    logits[4:] = np.arange(900) * 40
    got = check_sample(ck, logits, [65536, 65536, 0, 65536, (16 << 16) + 1, 2**32 - 1, 65536, 65536],
                       [2**32 - 1] * 8, [2**32 - 1] * 8, [0] * 8)
    assert got.token.tolist()[:3] == [-1, 899, 5] and got.kept.tolist()[:4] == [0, 1, 1, 200]
    check_sample(ck, logits, [0] * 8)
    check_sample(ck, logits, [65536] * 8, [5] * 8, [ONE // 2] * 8, [2**32 - 1] * 8)
    for random in (0, 1, 2**63, 2**64 - 1):
        check_sample(ck, logits, [65536] * 8, random=np.full(8, random, np.uint64))
        check_sample(ck, logits, [90000] * 8, [40] * 8, random=np.full(8, random, np.uint64))
    weights = [int(EXP[min(256 * (899 - i) * 40 // 65536, 4096)]) for i in range(900)]
    row = np.stack([np.arange(900) * 40] * 5).astype(np.int64)
    got = check_sample(ck, row, [65536] * 5, random=np.array([0, weights[0] - 1, weights[0], sum(weights) - 1, sum(weights)],
                                                             np.uint64))
    assert got.token.tolist() == [0, 0, 1, 899, 0]


def test_sampling_with_other_tables(ck):
    """A table that falls to zero, one of equal entries, one of zeros alone."""
    rng = np.random.default_rng(3)
    logits = (rng.standard_normal((30, 3000)) * 4 * 65536).astype(np.int64)
    t, k, p, m = settings(rng, 30, 3000)
    steep, flat = np.zeros(4097, np.uint32), np.full(4097, 2**30, np.uint32)
    steep[:300] = np.linspace(2**30, 1, 300).astype(np.uint32)
    for exp in (steep, flat):
        check_sample(ck, logits, t, k, p, m, exp=exp)
        check_sample(ck, logits, t, exp=exp)
    zeros = cuda(np.zeros(4097, np.int32))
    i32 = lambda a: cuda(np.array(a, np.uint32).view(np.int32))
    for args in ({}, dict(top_k=i32(k), top_p=i32(p), min_p=i32(m))):
        rc, got = ck.sample(cuda(logits), i32(np.maximum(t, 1)), cuda(np.arange(30)), zeros, **args)
        assert rc == 0 and ((got.token >= -1) & (got.token < 3000)).all()


def test_sampling_of_rows_beyond_32_bits_apart(ck):
    """Three rows of a matrix whose rows are 2^30 words apart, in blocks of their own and in clusters."""
    import torch
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 26 GB of device memory")
    rng = np.random.default_rng(6)
    wide = torch.empty(3, 2**30 + 3, dtype=torch.int64, device="cuda")
    for vocab in (700, 33000):
        wide[:, :vocab] = cuda((rng.standard_normal((3, vocab)) * 65536).astype(np.int64))
        check_sample(ck, wide[:, :vocab], [65536] * 3, [40, 0, 9], [ONE // 2] * 3, [0, 7, 0])
        check_sample(ck, wide[:, :vocab], [65536] * 3)


def test_sampling_of_rows_apart_on_other_streams_and_captured(ck):
    import torch
    rng = np.random.default_rng(4)
    wide = cuda((rng.standard_normal((11, 5011)) * 3 * 65536).astype(np.int64))
    t, k, p, m = settings(rng, 11, 5000)
    check_sample(ck, wide[:, 7:5007], t, k, p, m)
    check_sample(ck, wide[:, 7:8], t, k, p, m)
    u32 = lambda a: cuda(np.array(a, np.uint32).view(np.int32))
    random, exp, logits = cuda(rng.integers(-2**63, 2**63, 11)), cuda(EXP.view(np.int32)), wide[:, :5000].contiguous()
    args = dict(top_k=u32(k), top_p=u32(p), min_p=u32(m))
    rc, want = ck.sample(logits, u32(t), random, exp, **args)
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    temperature = u32(t)
    torch.cuda.synchronize()
    for turn in range(20):
        outs.append(ck.sample(logits, temperature, random, exp, stream=streams[turn % 2], **args))
    torch.cuda.synchronize()
    for rc, got in outs:
        assert rc == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    place = logits.clone()
    with torch.cuda.graph(graph):
        rc, got = ck.sample(place, temperature, random, exp, **args)
    place.copy_(logits.flip(1))
    graph.replay()
    rc, flipped = ck.sample(logits.flip(1).contiguous(), temperature, random, exp, **args)
    assert all(torch.equal(a, b) for a, b in zip(got, flipped))
    for bad in (dict(logits=logits[0]), dict(logits=logits.int()), dict(logits=logits.T), dict(temperature=temperature[:4]),
                dict(temperature=temperature.long()), dict(random=random[:4]), dict(exp_table=exp[:4096]),
                dict(top_k=temperature[:2]), dict(top_p=random), dict(min_p=temperature.cpu())):
        good = dict(logits=logits, temperature=temperature, random=random, exp_table=exp)
        good.update(bad)
        with pytest.raises(ValueError):
            ck.sample(**good)


# ---------------------------------------------------------------- together

class PlainStream:
    """One run of a model with a window a layer, position by position from the oracle's steps."""

    def __init__(self, spec, art, views):
        self.spec, self.views, self.keys = spec, views, [([], []) for _ in range(spec.layers)]
        self.tensor = lambda i: synth.artifact_tensor(art, i)

    def logits(self, token, pos):
        spec, T, hd = self.spec, self.tensor, self.spec.dim // self.spec.heads
        rope, inv, exp = T(synth.T_ROPE)[pos], synth.inv_sqrt_head(hd), T(synth.T_EXP)

        def turn(x):
            pairs = [oracle.rotate(int(x[h * hd + 2 * j]), int(x[h * hd + 2 * j + 1]), int(rope[j][0]), int(rope[j][1]))
                     for h in range(len(x) // hd) for j in range(hd // 2)]
            return np.array(pairs, np.int64).reshape(-1)

        x = oracle.embed(T(synth.T_EMBED)[token], int(T(synth.T_EMBED_SCALE)[token]))
        for l in range(spec.layers):
            W = lambda j: T(synth.GLOBAL_TENSORS + synth.PER_LAYER * l + j)
            a = oracle.rmsnorm(x, W(synth.L_ATTN_NORM))
            q, k, v = (oracle.matrow(W(w), W(s), a) for w, s in ((synth.L_WQ, synth.L_SQ), (synth.L_WK, synth.L_SK),
                                                                 (synth.L_WV, synth.L_SV)))
            q, k = turn(q), turn(k)
            K, V = self.keys[l]
            K.append(k.astype(np.int32))
            V.append(v.astype(np.int32))
            at, group = seen(pos, *self.views[l]), spec.heads // spec.kv_heads
            out = []
            for h in range(spec.heads):
                c = slice(h // group * hd, (h // group + 1) * hd)
                out.append(oracle.attention_head(q[h * hd:(h + 1) * hd], np.stack([K[t][c] for t in at]),
                                                 np.stack([V[t][c] for t in at]), inv, exp)[0])
            x = x + oracle.matrow(W(synth.L_WO), W(synth.L_SO), np.concatenate(out))
            a = oracle.rmsnorm(x, W(synth.L_FFN_NORM))
            g, u = oracle.matrow(W(synth.L_W1), W(synth.L_S1), a), oracle.matrow(W(synth.L_W3), W(synth.L_S3), a)
            x = x + oracle.matrow(W(synth.L_W2), W(synth.L_S2), oracle.silu_gate(g, u, T(synth.T_SILU)))
        return oracle.matrow(T(synth.T_CLS), T(synth.T_CLS_SCALE), oracle.rmsnorm(x, T(synth.T_FINAL_NORM)))


def test_the_plain_stream_is_the_oracle_without_windows():
    spec = synth.GQA
    art = synth.build_artifact(spec)
    ids = [int(t) for t in synth.prompt_ids(spec, 9)]
    plain = PlainStream(spec, art, [(0, 10**6)] * spec.layers)
    got = [plain.logits(t, i) for i, t in enumerate(ids)][-1]
    model = oracle.Model(art)
    rc, state = model.init_state(np.array(ids, np.uint32), 1)
    assert rc == 0 and model.turn(state, len(ids))[0] == 0
    at = model.layout(len(ids), 1)["logits"]
    assert np.array_equal(got, state[at:at + 8 * spec.vocab].view("<i8"))


@pytest.mark.parametrize("views", [[(4, 12)] * 5, [(0, 5)] * 5, [(2, 9), (0, 1), (4, 12), (1, 12), (0, 7)],
                                   [(4, 12), (0, 10**6), (0, 3), (4, 12), (4, 12)]], ids=str)
@pytest.mark.parametrize("captured", [False, True])
def test_streams_served_together(ck, views, captured):
    """Three prompts in ragged chunks, then token by token: the tables' step, the model's layers with a
    window each, and sampling, on the device from step to step; every token and the last logits are
    those of runs from the oracle's steps.  Captured, the steps by single tokens are one graph."""
    import torch
    spec = synth.GQA
    art = synth.build_artifact(spec)
    rc, model = ck.Model.load(art)
    assert rc == 0
    prompts = [[int(t) for t in synth.prompt_ids(spec, n, run=i)] for i, n in enumerate((23, 5, 31))]
    seqs, page, steps, stride = 3, 8, 16, 10
    whole = any(w > 100 for _, w in views)
    widest = None if whole else ck.Window(max(s for s, _ in views), max(w for _, w in views))
    pages = 14 if whole else 11  # (14 hold the three sequences' positions)
    windows = [ck.Window(*v) for v in views]
    cache = ck.PagedCache.empty(pages, spec.layers, spec.kv_heads, page, spec.dim // spec.heads)
    plan = ck.PagePlan(cache, seqs, stride)
    i32 = lambda a: cuda(np.array(a, np.int32))
    lens, table = i32([0] * seqs), i32(np.full((seqs, stride), -1))
    exp = model.exp_table()
    settings = dict(temperature=i32([60000, 0, 90000]), top_k=i32([0, 0, 40]), top_p=i32([ONE * 9 // 10, ONE, ONE]),
                    min_p=i32([0, 0, ONE // 50]))
    random = np.random.default_rng(8).integers(0, 2**64, (steps, seqs), dtype=np.uint64)
    # the prompts, in two chunks
    done = [0] * seqs
    for part in range(2):
        news = [len(p) // 2 if part == 0 else len(p) - len(p) // 2 for p in prompts]
        rc, got = plan.advance(lens, table, i32(news), sum(news), window=widest)
        assert rc == 0 and got.status.tolist() == [0] * seqs
        lens, table = got.lens, got.table
        tokens = [t for p, d, n in zip(prompts, done, news) for t in p[d:d + n]]
        done = [d + n for d, n in zip(done, news)]
        batch = ck.PagedBatch(table, lens, got.starts, None, sum(news), max(news), max(done))
        rc, logits = model.turn_paged(cache, batch, i32(tokens), window=windows)
        assert rc == 0 and batch.errors() == [None] * seqs
    # single tokens, all on the device
    draws, one = cuda(random.view(np.int64)), i32([1] * seqs)
    lens, table, logits, count = lens.clone(), table.clone(), logits.clone(), torch.zeros((), dtype=torch.int64, device="cuda")
    chosen, status = torch.zeros((steps, seqs), dtype=torch.int32, device="cuda"), torch.full((seqs,), -1, dtype=torch.int64, device="cuda")

    def step():
        rc, got = ck.sample(logits, settings["temperature"], draws.index_select(0, count[None])[0], exp, settings["top_k"],
                            settings["top_p"], settings["min_p"])
        assert rc == 0
        chosen.index_copy_(0, count[None], got.token[None])
        rc, grown = plan.advance(lens, table, one, seqs, window=widest)
        assert rc == 0
        lens.copy_(grown.lens)
        table.copy_(grown.table)
        batch = ck.PagedBatch(table, lens, grown.starts, status, seqs, 1, stride * page)
        rc, _ = model.turn_paged(cache, batch, got.token, logits=logits, window=windows)
        assert rc == 0
        count.add_(1)
        return grown

    if captured:
        keep = [t.clone() for t in (lens, table, logits, count, cache.k, cache.v)]
        grown = step()          # (loads every kernel)
        for t, old in zip((lens, table, logits, count, cache.k, cache.v), keep):
            t.copy_(old)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            grown = step()
        for _ in range(steps):
            graph.replay()
            assert grown.status.tolist() == [0] * seqs
    else:
        for _ in range(steps):
            assert step().status.tolist() == [0] * seqs
    assert status.tolist() == [-1] * seqs
    if not whole:
        assert (table == -1).sum() > seqs * (stride - 6)
    for i, prompt in enumerate(prompts):
        plain, ids = PlainStream(spec, art, views), list(prompt)
        for pos in range(len(prompt) + steps):
            want = plain.logits(ids[pos], pos)
            if pos >= len(prompt) - 1 and len(ids) < len(prompt) + steps:
                n = len(ids) - len(prompt)
                token, _, _ = plain_sample(want, *(int(settings[x][i]) for x in ("temperature", "top_k", "top_p", "min_p")),
                                           int(random[n, i]))
                ids.append(token)
        assert chosen[:, i].tolist() == ids[len(prompt):], i
        assert np.array_equal(logits[i].cpu().numpy(), want), i
