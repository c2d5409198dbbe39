"""The paged cache's operators and beam search on the GPU against plain integer implementations
(the CPU oracle's steps and Python's integers).  All of it is integer work: tolerance 0."""
import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu

MIN = -2**63
EXP = synth.exp_table()


@pytest.fixture(scope="module")
def ck():
    import torch
    import fixed_point_int8_gb300 as ck
    from fixed_point_int8_gb300 import build
    build.build()
    torch.cuda.init()
    return ck


def cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Setup:
    """A pool of random words, tables of scattered pages, and a batch's new rows."""

    def __init__(self, ck, lens, news, heads, kv_heads, hd, page, layers=2, seed=0, lead=0, tail=0, spare=3,
                 spread=2.0, max_len=None):
        import torch
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.news, self.heads, self.kv, self.hd, self.page = lens, news, heads, kv_heads, hd, page
        n_pages = [-(-n // page) for n in lens]
        stride = max(n_pages) + 1
        ids = rng.permutation(sum(n_pages) + spare)
        self.table = np.full((len(lens), stride), -1, np.int32)
        at = 0
        for i, n in enumerate(n_pages):
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.pages = len(ids)
        shape = (self.pages, layers, kv_heads, page, hd)
        self.k = (rng.standard_normal(shape) * spread * 65536).astype(np.int32)
        self.v = (rng.standard_normal(shape) * spread * 65536).astype(np.int32)
        self.starts = (np.cumsum([0] + list(news)) + lead).astype(np.int32)
        self.rows = int(self.starts[-1]) + tail
        self.cache = ck.PagedCache(cuda(self.k), cuda(self.v))
        self.batch = ck.PagedBatch(cuda(self.table), cuda(np.array(lens, np.int32)), cuda(self.starts), None,
                                   self.rows, max(max(news), 1), max_len or max(max(lens), 1))

    def words(self, pool, layer, s, kvh, n):
        """Positions 0 .. n-1 of sequence s as [n][hd]."""
        t = np.arange(n)
        return pool[self.table[s, t // self.page], layer, kvh, t % self.page]

    def attention(self, layer, q, inv, exp=EXP, fill=0):
        out = np.full((self.rows, self.heads * self.hd), fill, np.int64)
        for s, (n, length) in enumerate(zip(self.news, self.lens)):
            for j in range(n):
                row, pos = self.starts[s] + j, length - n + j
                for h in range(self.heads):
                    kvh, c = h // (self.heads // self.kv), slice(h * self.hd, (h + 1) * self.hd)
                    if pos < 0:
                        out[row, c] = 0
                        continue
                    out[row, c] = plain_attention(q[row, c], self.words(self.k, layer, s, kvh, pos + 1),
                                                  self.words(self.v, layer, s, kvh, pos + 1), inv, exp)
        return out


def plain_attention(q, K, V, inv, exp=EXP):
    """One head of one row with wrapping 64-bit words."""
    with np.errstate(over="ignore"):
        K, V = K.astype(np.int64), V.astype(np.int64)
        s = (((K * q[None, :]).sum(-1) >> 16) * np.int64(inv)) >> 24
        d = (np.uint64(int(s.max()) & (2**64 - 1)) - s.view(np.uint64)) >> np.uint64(8)
        e = exp[np.minimum(d, np.uint64(4096)).astype(np.int64)].astype(np.int64)
        p = (e << 24) // int(e.sum())
        return (p[:, None] * V).sum(0) >> 24


def test_plain_attention_is_the_oracles():
    rng = np.random.default_rng(3)
    for n, hd, spread in ((1, 4, 1), (37, 64, 65536), (5, 128, 2**31 - 1)):
        q = rng.integers(-2**20, 2**20, hd)
        K, V = (rng.integers(-spread, spread + 1, (n, hd)).astype(np.int32) for _ in range(2))
        want = oracle.attention_head(q, K, V, synth.inv_sqrt_head(hd), EXP)
        want = want[0] if isinstance(want, tuple) else want
        assert np.array_equal(plain_attention(q, K, V, synth.inv_sqrt_head(hd)), want)


# ---------------------------------------------------------------- attention

# lens, news, heads, kv heads, head, page: single tokens and chunks, one position, tables that end
# inside a page, shared key heads, a sequence without new rows, one with more rows than positions
ATTENTION = [
    ([1], [1], 1, 1, 4, 8),
    ([33], [1], 8, 4, 8, 16),
    ([1, 2, 15, 16, 17, 100], [1] * 6, 4, 4, 16, 16),
    ([257, 64], [1, 1], 8, 2, 64, 32),
    ([300], [1], 3, 3, 128, 256),
    ([1025], [1], 32, 32, 64, 64),
    ([2500], [1], 4, 1, 128, 16),
    ([0, 5, 9], [1, 0, 2], 2, 2, 32, 8),
    ([3], [5], 2, 1, 8, 8),
    ([130, 67], [130, 3], 4, 2, 64, 16),
    ([200], [200], 2, 2, 128, 32),
    ([77, 300, 12], [20, 129, 12], 4, 4, 32, 64),
    ([513], [65], 8, 1, 64, 64),
    ([700], [40], 6, 2, 16, 8),
    ([260], [129], 2, 2, 4, 16),
]
# work enough for the tensor-core tiles: shared key heads, ragged, a last tile of few queries, pages
# that end inside a block, rows without a position
TILES = [
    ([900, 333], [70, 129], 32, 8, 64, 16),
    ([640], [200], 16, 16, 128, 32),
    ([1030, 40], [129, 40], 8, 1, 64, 8),
    ([2100], [20], 32, 4, 128, 64),
    ([77, 130], [90, 2], 48, 3, 64, 32),
    ([300, 1000, 5], [0, 65, 5], 32, 32, 64, 256),
]


def on_tiles(ck, s):
    """The call takes the tensor-core tiles (their scores need scratch; short ones of a few queries
    need none)."""
    return ck.paged_attention_work(s.cache, s.batch, s.heads).numel() > 1 << 20


@pytest.mark.parametrize("lens,news,heads,kv,hd,page", ATTENTION + TILES)
def test_attention_against_the_plain_form(ck, lens, news, heads, kv, hd, page):
    s = Setup(ck, lens, news, heads, kv, hd, page, seed=hd + len(lens))
    assert on_tiles(ck, s) == ((lens, news, heads, kv, hd, page) in TILES)
    q = (s.rng.standard_normal((s.rows, heads * hd)) * 65536).astype(np.int64)
    inv = synth.inv_sqrt_head(hd)
    for layer in (0, 1):
        rc, out = ck.paged_attention(s.cache, layer, s.batch, cuda(q), cuda(EXP.view(np.int32)), inv)
        assert rc == 0
        assert np.array_equal(out.cpu().numpy(), s.attention(layer, q, inv))
    assert s.batch.errors() == [None] * len(lens)


@pytest.mark.parametrize("lens,news,heads,kv,hd,page", TILES)
def test_tiles_give_the_same_bits_every_time(ck, lens, news, heads, kv, hd, page):
    import torch
    s = Setup(ck, lens, news, heads, kv, hd, page, seed=hd + len(lens))
    assert on_tiles(ck, s)
    q, exp = cuda((s.rng.standard_normal((s.rows, heads * hd)) * 65536).astype(np.int64)), cuda(EXP.view(np.int32))
    inv = synth.inv_sqrt_head(hd)
    rc, first = ck.paged_attention(s.cache, 0, s.batch, q, exp, inv)
    assert rc == 0
    for _ in range(100):
        rc, out = ck.paged_attention(s.cache, 0, s.batch, q, exp, inv)
        assert rc == 0 and torch.equal(out, first)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("q_spread,kv_spread", [(2**62, 65536), (65536, 2**31 - 1), (2**31, 2**31 - 1),
                                                (2**22, 2**23), (2**23 + 5, 2**23 + 5), (1, 1), (0, 65536)])
def test_attention_over_the_whole_range_of_values(ck, new, q_spread, kv_spread):
    """Queries to 63 bits and cached words to 32, wrapping products among them."""
    s = Setup(ck, [150], [new], 4, 2, 64, 16, seed=1) if new == 1 else Setup(ck, [600], [new], 32, 4, 64, 16, seed=1)
    assert on_tiles(ck, s) == (new == 70)
    s.k[:] = s.rng.integers(-kv_spread - 1, kv_spread + 1, s.k.shape)
    s.v[:] = s.rng.integers(-kv_spread - 1, kv_spread + 1, s.v.shape)
    s.cache.k.copy_(cuda(s.k))
    s.cache.v.copy_(cuda(s.v))
    q = s.rng.integers(-q_spread, q_spread + 1, (s.rows, s.heads * 64))
    inv = synth.inv_sqrt_head(64)
    rc, out = ck.paged_attention(s.cache, 1, s.batch, cuda(q), cuda(EXP.view(np.int32)), inv)
    assert rc == 0
    assert np.array_equal(out.cpu().numpy(), s.attention(1, q, inv))


@pytest.mark.parametrize("new", [1, 130])
def test_attention_with_equal_and_with_single_scores(ck, new):
    """Every score the same, and one score far above all others (its probability is 2^24)."""
    s = Setup(ck, [200], [new], 2, 2, 64, 16, seed=2) if new == 1 else Setup(ck, [400], [new], 32, 4, 64, 16, seed=2)
    assert on_tiles(ck, s) == (new == 130)
    inv = synth.inv_sqrt_head(64)
    exp = EXP.copy()
    exp[4096] = 0
    for kind in ("equal", "single"):
        s.k[:] = 0
        if kind == "single":
            s.k[s.table[0, 0], :, :, 3] = 1 << 20
        s.cache.k.copy_(cuda(s.k))
        q = np.full((s.rows, s.heads * 64), 1 << 18, np.int64)
        rc, out = ck.paged_attention(s.cache, 0, s.batch, cuda(q), cuda(exp.view(np.int32)), inv)
        assert rc == 0
        assert np.array_equal(out.cpu().numpy(), s.attention(0, q, inv, exp))


@pytest.mark.parametrize("hd,new,length,heads,kv", [(64, 70, 600, 32, 4), (128, 33, 777, 32, 8), (64, 1, 300, 2, 1)])
def test_attention_at_the_ends_of_three_digits(ck, hd, new, length, heads, kv):
    """Words at both ends of what three balanced 8-bit digits hold, in every combination of signs:
    the largest sums that the tensor cores' f32 accumulators see."""
    lo, hi = -128 * 65793, 127 * 65793
    s = Setup(ck, [length], [new], heads, kv, hd, 16, seed=hd)
    assert on_tiles(ck, s) == (new > 1)
    inv = synth.inv_sqrt_head(hd)
    for kind in ("all low", "all high", "mixed", "equal scores"):
        pick = {"all low": [lo], "all high": [hi], "mixed": [lo, hi], "equal scores": [lo]}[kind]
        s.k[:] = s.rng.choice(pick, s.k.shape)
        s.v[:] = s.rng.choice([lo, hi] if kind == "equal scores" else pick, s.v.shape)
        s.cache.k.copy_(cuda(s.k))
        s.cache.v.copy_(cuda(s.v))
        q = s.rng.choice(pick, (s.rows, heads * hd)).astype(np.int64)
        rc, out = ck.paged_attention(s.cache, 0, s.batch, cuda(q), cuda(EXP.view(np.int32)), inv)
        assert rc == 0
        assert np.array_equal(out.cpu().numpy(), s.attention(0, q, inv)), kind


@pytest.mark.parametrize("inv", [1, 1 << 21, (1 << 24) + 1, 2**32 - 1])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_with_other_scales(ck, inv, new):
    """One over the square root may be any u32: products and scores that pass 32 bits."""
    s = Setup(ck, [300], [new], 2, 2, 64, 16, seed=3) if new == 1 else Setup(ck, [600], [new], 32, 4, 64, 16, seed=3)
    assert on_tiles(ck, s) == (new == 40)
    q = (s.rng.standard_normal((s.rows, s.heads * 64)) * 65536 * 8).astype(np.int64)
    rc, out = ck.paged_attention(s.cache, 1, s.batch, cuda(q), cuda(EXP.view(np.int32)), inv)
    assert rc == 0
    assert np.array_equal(out.cpu().numpy(), s.attention(1, q, inv))


def test_attention_of_a_long_sequence_of_few_heads(ck):
    """Clusters of sixteen blocks, scores in the scratch, and a bound far above the length."""
    for lens, max_len in (([9001], 9001), ([40, 7], 200000)):
        s = Setup(ck, lens, [1] * len(lens), 4, 1, 64, 32, seed=4, max_len=max_len)
        s.table = np.concatenate([s.table, np.full((len(lens), max_len // 32 + 2), -1, np.int32)], 1)
        s.batch = ck.PagedBatch(cuda(s.table), cuda(np.array(lens, np.int32)), cuda(s.starts), None, s.rows, 1, max_len)
        q = (s.rng.standard_normal((s.rows, 256)) * 65536).astype(np.int64)
        rc, out = ck.paged_attention(s.cache, 0, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 21)
        assert rc == 0
        assert np.array_equal(out.cpu().numpy(), s.attention(0, q, 1 << 21))


def test_pools_beyond_32_bits_of_words(ck):
    """Stores, attention (both forms), a fork and packing at the far end of pools of over 2^32
    words each."""
    import torch
    page, hd, pages = 256, 128, 131072 + 64
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 36 GB of device memory")
    cache = ck.PagedCache.empty(pages, 1, 1, page, hd)
    rng = np.random.default_rng(8)
    n, top = 300, pages - 1
    table = np.full((1, 4), -1, np.int32)
    table[0, :2] = [top, top - 40]
    k, v = ((rng.standard_normal((n, hd)) * 65536).astype(np.int64) for _ in range(2))
    q = (rng.standard_normal((n, 32 * hd)) * 65536).astype(np.int64)
    batch = ck.PagedBatch(cuda(table), cuda(np.array([n], np.int32)), cuda(np.array([0, n], np.int32)), None, n, n, n)
    rc, rotated = ck.paged_store(cache, 0, batch, cuda(q), cuda(k), cuda(v), cuda(rope_of(n, 0)))
    assert rc == 0 and batch.errors() == [None] and np.array_equal(rotated.cpu().numpy(), q)
    inv = synth.inv_sqrt_head(hd)
    assert ck.paged_attention_work(cache, batch, 32).numel() > 1 << 20       # the tiles
    rc, out = ck.paged_attention(cache, 0, batch, rotated, cuda(EXP.view(np.int32)), inv)
    assert rc == 0
    for row in (0, 130, 299):
        for h in (0, 17, 31):
            want = plain_attention(q[row, h * hd:(h + 1) * hd], k[:row + 1], v[:row + 1], inv)
            assert np.array_equal(out[row, h * hd:(h + 1) * hd].cpu().numpy(), want)
    plan = ck.PagePlan(cache, 2, 4)
    held = torch.ones(pages, dtype=torch.uint8, device="cuda")
    held[top - 7] = 0
    rc, fork = plan.fork(cuda(np.array([0, 0], np.int32)), batch.lens, batch.table, cuda(np.array([0, 0], np.int32)), held=held)
    assert rc == 0 and fork.status.tolist() == [0, 0]
    assert fork.table.tolist() == [[top, top - 40, -1, -1], [top, top - 7, -1, -1]]
    rc, packed = plan.compact(fork.lens, fork.table)
    assert rc == 0 and int(packed.used) == 3 and packed.table.tolist() == [[2, 0, -1, -1], [2, 1, -1, -1]]
    one = ck.PagedBatch(packed.table, fork.lens, cuda(np.array([0, 1, 2], np.int32)), None, 2, 1, n)
    rc, last = ck.paged_attention(cache, 0, one, rotated[[299, 299]].contiguous(), cuda(EXP.view(np.int32)), inv)
    assert rc == 0
    assert torch.equal(last[0], out[299]) and torch.equal(last[1], out[299])


def test_calls_on_two_streams_and_captured_ones_repeat(ck):
    """Attention, both forms, on two streams at once with scratch of their own; and captured, then
    replayed over other inputs in the same places."""
    import torch
    jobs = []
    for new in (1, 60):
        s = Setup(ck, [500, 420], [new, new], 32, 4, 64, 16, seed=new)
        assert on_tiles(ck, s) == (new == 60)
        q = [(s.rng.standard_normal((s.rows, 32 * 64)) * 65536).astype(np.int64) for _ in range(2)]
        jobs.append((s, q, [s.attention(0, x, 1 << 21) for x in q]))
    exp = cuda(EXP.view(np.int32))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    dev = [[cuda(x) for x in q] for _, q, _ in jobs]
    torch.cuda.synchronize()
    outs = []
    for turn in range(20):
        for (s, _, _), d, stream in zip(jobs, dev, streams):
            outs.append(ck.paged_attention(s.cache, 0, s.batch, d[turn % 2], exp, 1 << 21, stream=stream))
    torch.cuda.synchronize()
    for i, (rc, out) in enumerate(outs):
        assert rc == 0 and np.array_equal(out.cpu().numpy(), jobs[i % 2][2][i // 2 % 2])
    for (s, q, want), d in zip(jobs, dev):
        place, out = d[0].clone(), torch.zeros_like(d[0])
        work = ck.paged_attention_work(s.cache, s.batch, 32)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rc, _ = ck.paged_attention(s.cache, 0, s.batch, place, exp, 1 << 21, out=out, work=work)
        assert rc == 0
        for turn in (1, 0, 1):
            place.copy_(d[turn])
            out.zero_()
            graph.replay()
            assert np.array_equal(out.cpu().numpy(), want[turn])


def test_inputs_freed_after_a_call_on_another_stream_stay_in_use(ck):
    """The stream is busy when the call is enqueued; its inputs are dropped and their memory asked
    for again on the current stream before the kernels run."""
    import torch
    s = Setup(ck, [70], [1], 4, 2, 64, 16)
    q = (s.rng.standard_normal((1, 256)) * 65536).astype(np.int64)
    want = s.attention(0, q, 1 << 21)
    side = torch.cuda.Stream()
    place, exp = cuda(q), cuda(EXP.view(np.int32))
    for t in (place, exp):  # (every kernel below is loaded before the stream is busy)
        torch.full_like(t, 3)
    ck.paged_attention(s.cache, 0, s.batch, place, exp, 1 << 21, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    rc, out = ck.paged_attention(s.cache, 0, s.batch, place, exp, 1 << 21, stream=side)
    assert rc == 0
    del place, exp
    other = [torch.full((1, 256), 3, dtype=torch.int64, device="cuda") for _ in range(500)]
    other += [torch.full((4097,), 3, dtype=torch.int32, device="cuda") for _ in range(100)]
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want) and len(other) == 600


def test_attention_leaves_rows_of_no_sequence_and_strided_queries(ck):
    """Rows before the first sequence and behind the last stay as they were; queries are a
    column range of wider rows."""
    import torch
    s = Setup(ck, [40, 90], [2, 3], 4, 2, 32, 8, lead=2, tail=3)
    wide = (s.rng.standard_normal((s.rows, 300)) * 65536).astype(np.int64)
    q = cuda(wide)[:, 64:192]
    out = torch.full((s.rows, 128), 7, dtype=torch.int64, device="cuda")
    rc, got = ck.paged_attention(s.cache, 0, s.batch, q, cuda(EXP.view(np.int32)), 1 << 21, out=out)
    assert rc == 0 and got is out
    assert np.array_equal(out.cpu().numpy(), s.attention(0, wide[:, 64:192], 1 << 21, fill=7))


# ---------------------------------------------------------------- stores

def plain_store(s, layer, q, k, v, rope, half):
    """Rotated queries, pools and first failures."""
    rot, hd = 2 * rope.shape[1], s.hd
    pairs = [(j, j + rot // 2) if half else (2 * j, 2 * j + 1) for j in range(rot // 2)]
    qo, pk, pv = np.zeros_like(q), s.k.copy(), s.v.copy()
    status = [None] * len(s.lens)

    def turn(x, pos):
        y = [int(w) for w in x]
        for j, (a, b) in enumerate(pairs):
            y[a], y[b] = oracle.rotate(int(x[a]), int(x[b]), int(rope[pos, j, 0]), int(rope[pos, j, 1]))
        return y

    def i32(w):
        return (w + 2**31) % 2**32 - 2**31

    for i, (n, length) in enumerate(zip(s.news, s.lens)):
        for j in range(n):
            row, pos = s.starts[i] + j, length - n + j
            if pos < 0:
                continue
            fails = []
            for h in range(s.heads):
                qo[row, h * hd:(h + 1) * hd] = turn(q[row, h * hd:(h + 1) * hd], pos)
            for h in range(s.kv):
                raw = [int(w) for w in k[row, h * hd:(h + 1) * hd]]
                fails += [(pos, layer, 6, h * hd + e) for e, w in enumerate(raw) if i32(w) != w]
                fails += [(pos, layer, 7, h * hd + e) for e, w in enumerate(v[row, h * hd:(h + 1) * hd])
                          if i32(int(w)) != w]
                turned = turn([i32(w) for w in raw], pos)
                fails += [(pos, layer, 8, h * hd + e) for e, w in enumerate(turned) if i32(w) != w]
                at = s.table[i, pos // s.page], layer, h, pos % s.page
                pk[at] = [i32(w) for w in turned]
                pv[at] = [i32(int(w)) for w in v[row, h * hd:(h + 1) * hd]]
            if fails:
                status[i] = min(fails + ([status[i]] if status[i] else []))
    return qo, pk, pv, status


def rope_of(positions, rot, base=10000.0, stretch=1.0, magnitude=1.0):
    """Angles of positions divided by `stretch`, cosine and sine times a magnitude."""
    angle = np.arange(positions)[:, None] / stretch * base**(-np.arange(0, rot, 2) / max(rot, 1))
    return np.rint(np.stack((np.cos(angle), np.sin(angle)), -1) * magnitude * 2**24).astype(np.int32)


STORE = [
    ([1], [1], 1, 1, 4, 8, 4, False, {}),
    ([133], [1], 32, 32, 128, 16, 128, False, {}),
    ([50, 7, 31], [50, 0, 9], 8, 4, 8, 16, 8, True, {}),
    ([40, 64], [33, 64], 6, 2, 64, 32, 32, True, {}),
    ([40, 64], [33, 64], 6, 2, 64, 32, 48, False, {"stretch": 4.0, "magnitude": 1.1386}),
    ([17], [17], 4, 1, 16, 8, 0, False, {}),
    ([3, 9], [5, 2], 2, 2, 32, 8, 32, True, {"base": 500000.0}),
]


@pytest.mark.parametrize("lens,news,heads,kv,hd,page,rot,half,scaled", STORE)
def test_store_against_the_plain_form(ck, lens, news, heads, kv, hd, page, rot, half, scaled):
    s = Setup(ck, lens, news, heads, kv, hd, page, seed=rot, lead=1, tail=2)
    cols = (heads + 2 * kv) * hd
    qkv = (s.rng.standard_normal((s.rows, cols)) * 65536).astype(np.int64)
    rope = rope_of(max(lens), rot, **scaled)
    parts = np.split(qkv, [heads * hd, (heads + kv) * hd], axis=1)
    import torch
    out = torch.zeros(s.rows, heads * hd, dtype=torch.int64, device="cuda")
    dev = cuda(qkv).split((heads * hd, kv * hd, kv * hd), -1)
    rc, q = ck.paged_store(s.cache, 1, s.batch, *dev, cuda(rope), half=half, out=out)
    assert rc == 0
    qo, pk, pv, status = plain_store(s, 1, *parts, rope, half)
    assert np.array_equal(q.cpu().numpy(), qo)
    assert np.array_equal(s.cache.k.cpu().numpy(), pk) and np.array_equal(s.cache.v.cpu().numpy(), pv)
    assert s.batch.errors() == status == [None] * len(lens)


@pytest.mark.parametrize("half", [False, True])
def test_store_reports_the_first_word_that_does_not_fit(ck, half):
    s = Setup(ck, [20, 30, 40], [20, 6, 4], 2, 2, 16, 8)
    q, k, v = ((s.rng.standard_normal((s.rows, 32)) * 65536).astype(np.int64) for _ in range(3))
    k[3, 5] = 2**31            # a key before its rotation, position 3 of the first sequence
    v[3, 1] = -2**31 - 1       # a value of the same position
    k[2, 8:12] = 2**31 - 1     # fits, but not every rotation of it does
    v[21, 31] = 2**40          # position 25 of the second
    v[26, :] = 2**31 - 1       # the third fits exactly
    q[4] = 2**62
    rope = rope_of(40, 16)
    rc, out = ck.paged_store(s.cache, 0, s.batch, cuda(q), cuda(k), cuda(v), cuda(rope), half=half)
    qo, pk, pv, status = plain_store(s, 0, q, k, v, rope, half)
    assert rc == 0 and status[0] and status[1] == (25, 0, 7, 31) and status[2] is None
    assert s.batch.errors() == status
    assert np.array_equal(out.cpu().numpy(), qo) and np.array_equal(s.cache.k.cpu().numpy(), pk)
    assert np.array_equal(s.cache.v.cpu().numpy(), pv)


# ---------------------------------------------------------------- sequences and pages that do not fit

def test_bad_pages_and_sequences_on_tiles(ck):
    """As below for the tensor-core tiles: a bad page reads as zeros, a sequence beyond the bounds is
    left as it was, one with words beyond the digits beside others is done all the same."""
    import torch
    s = Setup(ck, [500, 480, 450, 470], [40, 40, 30, 40], 32, 4, 64, 16, seed=7)
    assert on_tiles(ck, s)
    s.v[s.table[2, 3]] = 2**31 - 1                       # beyond the digits
    s.k[s.table[3, 1]] = 2**30
    s.cache.k.copy_(cuda(s.k))
    s.cache.v.copy_(cuda(s.v))
    q = (s.rng.standard_normal((s.rows, 2048)) * 65536).astype(np.int64)
    s.batch.lens.copy_(cuda(np.array([500, 501, 450, 470], np.int32)))   # the second is past max_len
    s.batch.table[0, 5] = s.pages + 3                    # positions 80 .. 95 of the first
    out = torch.full((s.rows, 2048), 5, dtype=torch.int64, device="cuda")
    rc, _ = ck.paged_attention(s.cache, 1, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 21, out=out)
    assert rc == 0
    assert s.batch.errors() == [(80, 1, 2, 0), (0, 1, 1, 0), None, None]
    for pool in (s.k, s.v):
        pool[s.table[0, 5]] = 0
    want, got = s.attention(1, q, 1 << 21), out.cpu().numpy()
    keep = np.r_[0:40, 80:150]
    assert np.array_equal(got[keep], want[keep]) and (got[40:80] == 5).all()


def test_bad_sequences_and_pages_are_reported_and_the_others_done(ck):
    """A length beyond the launch's bound, a table entry outside the pool, a position past the
    rotary table: nothing outside the pool is touched, and the other sequences come out right."""
    import torch
    s = Setup(ck, [20, 30, 25, 12], [2, 2, 2, 2], 2, 2, 16, 8)
    q = (s.rng.standard_normal((s.rows, 32)) * 65536).astype(np.int64)
    kv = [(s.rng.standard_normal((s.rows, 32)) * 65536).astype(np.int64) for _ in range(2)]
    want = s.attention(0, q, 1 << 22, fill=5)
    lens = np.array([20, 31, 25, 12], np.int32)          # the second is past max_len
    table = s.table.copy()
    table[2, 1] = s.pages                                 # positions 8 .. 15 of the third
    s.batch.lens.copy_(cuda(lens))
    s.batch.table.copy_(cuda(table))
    out = torch.full((s.rows, 32), 5, dtype=torch.int64, device="cuda")
    rc, _ = ck.paged_attention(s.cache, 0, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 22, out=out)
    assert rc == 0
    got = out.cpu().numpy()
    assert np.array_equal(got[[0, 1, 6, 7]], want[[0, 1, 6, 7]]) and (got[2:4] == 5).all()
    assert s.batch.errors() == [None, (0, 0, 1, 0), (8, 0, 2, 0), None]
    # the words of a page outside the pool read as zeros
    k, v = s.k.copy(), s.v.copy()
    for pool in (k, v):
        pool[s.table[2, 1]] = 0
    s.k, s.v = k, v
    assert np.array_equal(got[4:6], s.attention(0, q, 1 << 22)[4:6])
    s.batch.status.fill_(-1)
    table[3, 1] = 2**31 - 1                               # positions 8 .. 15 of the fourth
    s.batch.table.copy_(cuda(table))
    before = s.cache.k.clone(), s.cache.v.clone()
    rc, _ = ck.paged_store(s.cache, 0, s.batch, cuda(q), cuda(kv[0]), cuda(kv[1]), cuda(rope_of(24, 16)))
    assert rc == 0
    assert s.batch.errors() == [None, (0, 0, 1, 0), (24, 0, 1, 0), (10, 0, 2, 0)]
    changed = {int(p) for p in torch.nonzero((s.cache.k != before[0]).flatten(1).any(1)).flatten()}
    assert changed == {int(s.table[0, 2]), int(s.table[2, 2])}


# ---------------------------------------------------------------- page tables

def plain_fork(lens, table, parent, grow, pages, page, held=()):
    rows, stride = len(parent), table.shape[1]
    status, kept, old = [0] * rows, [[] for _ in range(rows)], [None] * rows
    for r, p in enumerate(parent):
        if p == -1:
            continue
        if not 0 <= p < len(lens):
            status[r] = 3
            continue
        n = int(lens[p])
        if n + int(grow[r]) > min(stride * page, 2**20 - 1):
            status[r] = 7
            continue
        if any(not 0 <= w < pages for w in table[p][:-(-n // page)]):
            status[r] = 3
            continue
        old[r] = n
        kept[r] = [int(w) for w in table[p][:n // page]]
    used = {w for row in kept for w in row}
    holder = {}
    for r in range(rows):
        if old[r] is not None and old[r] % page:
            holder.setdefault(int(table[parent[r]][old[r] // page]), r)
    for w, r in holder.items():
        if w not in used:
            kept[r].append(w)
    free = [w for w in range(pages) if w not in used and w not in holder and w not in set(held)]
    asked, copies, out_lens = 0, [], [0] * rows
    for r in range(rows):
        if old[r] is None:
            continue
        need = -(-(old[r] + int(grow[r])) // page) - len(kept[r])
        mine = free[asked:asked + need]
        asked += need
        if len(mine) < need:
            status[r], kept[r] = 4, []
            continue
        if old[r] % page and len(kept[r]) == old[r] // page:
            copies.append((int(table[parent[r]][old[r] // page]), mine[0], old[r] % page))
        kept[r] += mine
        out_lens[r] = old[r] + int(grow[r])
    out = np.full((rows, stride), -1, np.int32)
    for r in range(rows):
        out[r, :len(kept[r])] = kept[r]
    return out, out_lens, status, copies


def check_fork(ck, k, v, lens, table, parent, grow, page, held=None):
    pages = k.shape[0]
    cache = ck.PagedCache(cuda(k), cuda(v))
    plan = ck.PagePlan(cache, max(len(parent), 1), table.shape[1])
    h = None if held is None else cuda(np.isin(np.arange(pages), held).astype(np.uint8))
    rc, got = plan.fork(cuda(np.array(parent, np.int32)), cuda(np.array(lens, np.int32)),
                        cuda(table.astype(np.int32)), cuda(np.array(grow, np.int32)), held=h)
    assert rc == 0
    out, out_lens, status, copies = plain_fork(lens, table, parent, grow, pages, page, held or ())
    assert got.status.tolist() == status
    assert got.lens.tolist() == out_lens
    assert np.array_equal(got.table.cpu().numpy(), out)
    for src, dst, n in copies:
        k[dst, :, :, :n], v[dst, :, :, :n] = k[src, :, :, :n], v[src, :, :, :n]
    assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
    return out, out_lens


def pools(rng, pages, layers, kv, page, hd):
    return [rng.integers(-2**31, 2**31, (pages, layers, kv, page, hd)).astype(np.int32) for _ in range(2)]


def test_fork_shares_copies_frees_and_grows(ck):
    rng = np.random.default_rng(5)
    page = 8
    k, v = pools(rng, 40, 3, 2, page, 16)
    table = np.full((4, 9), -1)
    lens = [21, 16, 5, 0]
    table[0, :3], table[1, :2], table[2, :1] = [30, 2, 7], [30, 9], [11]
    # three children of row 0, one of row 1 (its pages are whole), none of row 2, one of the empty row,
    # an empty row, a parent that does not exist
    parent, grow = [0, 1, 0, 0, 3, -1, 4], [1, 1, 4, 50, 9, 3, 1]
    check_fork(ck, k, v, lens, table, parent, grow, page)
    # a page that is whole for one row and part-filled for another: every part-filled row copies
    table[1, 1] = 7
    check_fork(ck, k, v, lens, table, [0, 1, 0], [0, 0, 1], page)
    # too long, and a table entry outside the pool
    table[2, 0] = 40
    check_fork(ck, k, v, lens, table, [0, 2, 1], [52, 1, 1], page)
    # pages of others, and a pool that runs out in the middle
    table[2, 0] = 11
    check_fork(ck, k, v, lens, table, [0, 0, 2, 1], [1, 1, 40, 1], page, held=list(range(12, 38)))


@pytest.mark.parametrize("seed", range(6))
def test_fork_step_after_step(ck, seed):
    """A search's reordering over many steps: tables and pools follow the plain form, and every
    row's cache reads as its ancestors wrote it."""
    rng = np.random.default_rng(seed)
    page, layers, kv, hd = [(8, 1, 1, 4), (16, 2, 3, 8), (32, 1, 2, 64), (8, 3, 1, 128), (16, 5, 4, 8), (64, 1, 1, 16)][seed]
    rows = [4, 70, 33, 1, 1100, 8][seed]
    stride, pages = 40 // page + 3, rows * 4 + 40
    k, v = pools(rng, pages, layers, kv, page, hd)
    table, lens = np.full((rows, stride), -1), [0] * rows
    parent = list(range(rows))
    for step in range(5):
        grow = [int(rng.integers(0, 8)) for _ in range(rows)]
        table, lens = check_fork(ck, k, v, lens, table, parent, grow, page)
        parent = [int(p) for p in rng.integers(-1, rows, rows)]


def test_compact_packs_the_pages_in_use(ck):
    rng = np.random.default_rng(6)
    page = 8
    for pages, rows, share in ((40, 5, True), (5000, 300, False), (1, 1, False), (64, 2, False), (6000, 1100, True),
                               (70000, 40, False)):
        k, v = pools(rng, pages, 2, 1, page, 8)
        stride = 6
        lens = [int(rng.integers(0, page * stride + 1)) for _ in range(rows)]
        if pages == 1:
            lens = [3]
        table, ids = np.full((rows, stride), -1, np.int32), rng.permutation(pages)
        at = 0
        for r in range(rows):
            n = -(-lens[r] // page)
            table[r, :n] = ids[at:at + n]
            at += n
        if share:
            table[1, :], lens[1] = table[0, :], lens[0]
            lens[2] = page * stride + 1                    # too long
            table[4, 0], lens[4] = pages, max(1, lens[4])  # outside the pool
        cache = ck.PagedCache(cuda(k), cuda(v))
        rc, got = ck.PagePlan(cache, rows, stride).compact(cuda(np.array(lens, np.int32)), cuda(table))
        assert rc == 0
        status = [0] * rows
        if share:
            status[2], status[4] = 7, 3
        mine = [[int(w) for w in table[r][:-(-lens[r] // page)]] if not status[r] else [] for r in range(rows)]
        used = sorted({w for row in mine for w in row})
        low = [w for w in range(len(used)) if w not in set(used)]
        to = {w: w for w in used if w < len(used)}
        to.update(zip([w for w in used if w >= len(used)], low))
        want = np.full((rows, stride), -1, np.int32)
        for r in range(rows):
            want[r, :len(mine[r])] = [to[w] for w in mine[r]]
        for src, dst in to.items():
            k[dst], v[dst] = k[src], v[src]
        assert got.status.tolist() == status and int(got.used) == len(used)
        assert np.array_equal(got.table.cpu().numpy(), want)
        assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)


# ---------------------------------------------------------------- beam search

LN2 = 744261118


def plain_log_sum(z):
    z = max(z, 2**30)
    n = z.bit_length() - 31
    y = z >> n
    t = ((y - 2**30) << 30) // (y + 2**30)
    square, c = (t * t) >> 30, 0
    for i in range(7, -1, -1):
        c = (2**31 // (2 * i + 1) + 1) // 2 + ((c * square) >> 30)
    return (n * LN2 + 2 * ((t * c) >> 30) + 2**13) >> 14


def plain_beam(logits, scores, done, groups, beams, done_token, stop):
    out = []
    vocab = logits.shape[1]
    for g in range(groups):
        found = []
        for r in range(g * beams, (g + 1) * beams):
            old = int(scores[r])
            if not -2**61 < old < 2**61:
                continue
            if done[r]:
                found.append((-old, r, vocab))
                continue
            row = logits[r].astype(object)
            d = np.minimum(max(row) - row, 2**62)
            z = sum(int(EXP[min(int(x) >> 8, 4096)]) for x in d)
            near = sorted(range(vocab), key=lambda i: (d[i], i))[:beams]
            found += [(int(d[i]) + plain_log_sum(z) - old, r, i) for i in near]
        found = sorted(found)[:beams]
        for cost, r, i in found:
            ended = i == vocab or (stop and i in (1, 2))
            out.append((-cost, r, done_token if i == vocab else i, int(ended)))
        out += [(MIN, -1, done_token, 0)] * (beams - len(found))
    return out


def check_beam(ck, logits, scores, done, groups, beams, done_token=0, stop=True, stride=None):
    vocab = logits.shape[1]
    dev = cuda(logits)
    if stride:
        import torch
        wide = torch.full((logits.shape[0], stride), 2**63 - 1, dtype=torch.int64, device="cuda")
        wide[:, :vocab] = dev
        dev = wide[:, :vocab]
    rc, got = ck.BeamPlan(groups, beams, vocab).select(dev, cuda(np.array(scores, np.int64)),
                                                       cuda(np.array(done, np.uint8)), cuda(EXP.view(np.int32)),
                                                       stop_tokens=stop, done_token=done_token)
    assert rc == 0
    got = list(zip(got.scores.tolist(), got.parent.tolist(), got.token.tolist(), got.done.tolist()))
    assert got == plain_beam(logits, scores, done, groups, beams, done_token, stop)


@pytest.mark.parametrize("groups,beams,vocab", [(1, 1, 1), (1, 4, 3), (2, 3, 7), (1, 4, 512), (3, 8, 1000), (2, 64, 333),
                                                (5, 5, 4099), (1, 33, 20011), (2, 2, 32000), (1, 1, 32000)])
def test_beam_selection_against_the_plain_form(ck, groups, beams, vocab):
    rng = np.random.default_rng(beams + vocab)
    rows = groups * beams
    logits = (rng.standard_normal((rows, vocab)) * 3 * 65536).astype(np.int64)
    scores = -rng.integers(0, 10 << 16, rows)
    check_beam(ck, logits, scores, np.zeros(rows), groups, beams)
    done = rng.random(rows) < 0.3
    scores[rng.random(rows) < 0.2] = MIN
    check_beam(ck, logits, scores, done, groups, beams, done_token=vocab - 1, stop=False)
    check_beam(ck, logits // 65536, scores, done, groups, beams, stride=vocab + 3)     # many ties


def test_beam_selection_at_the_edges(ck):
    """All logits equal, extremes of 64 bits, the first step (one live beam), a search of dead
    beams, scores at the bounds, ascending and descending logits."""
    rng = np.random.default_rng(9)
    for vocab in (40, 5000):
        check_beam(ck, np.zeros((4, vocab), np.int64), [0, -5, -5, -10**9], [0, 0, 0, 0], 1, 4)
        logits = rng.integers(-2**63, 2**63, (8, vocab))
        logits[0, 5], logits[0, 7], logits[1, :] = 2**63 - 1, MIN, MIN
        check_beam(ck, logits, [0, MIN, MIN, MIN, 2**61, -2**61, 2**61 - 1, 1 - 2**61], [0] * 8, 2, 4)
        check_beam(ck, logits, [MIN] * 4 + [0] * 4, [0, 1, 0, 1] * 2, 2, 4)
        ramp = np.arange(vocab)[None, :] * np.array([1, -1, 300, -300])[:, None]
        check_beam(ck, ramp.astype(np.int64), [0, 0, 0, 0], [0] * 4, 1, 4)
        check_beam(ck, ramp.astype(np.int64), [0, 0, 0, 0], [0] * 4, 4, 1)


@pytest.mark.parametrize("groups,beams,vocab", [(256, 8, 5000), (700, 3, 4096), (64, 8, 32000)])
def test_rows_that_follow_one_another_in_a_cluster(ck, groups, beams, vocab):
    """More rows than clusters are resident, rows of far apart and of close logits in turn: a block's
    counts of one row are not another's.  The same bits every time, and the plain form's in some."""
    import torch
    rng = np.random.default_rng(vocab)
    rows = groups * beams
    logits = (rng.standard_normal((rows, vocab)) * np.array([1, 65536, 2.0**40])[np.arange(rows) % 3, None]).astype(np.int64)
    scores, done = -rng.integers(0, 10 << 16, rows), np.zeros(rows, np.uint8)
    done[::7] = 1
    plan = ck.BeamPlan(groups, beams, vocab)
    dev = cuda(logits), cuda(scores), cuda(done), cuda(EXP.view(np.int32))
    rc, first = plan.select(*dev)
    assert rc == 0
    for _ in range(100):
        rc, again = plan.select(*dev)
        assert rc == 0 and all(torch.equal(a, b) for a, b in zip(first, again))
    for g in (0, groups // 2, groups - 1):
        at = slice(g * beams, (g + 1) * beams)
        want = plain_beam(logits[at], scores[at], done[at], 1, beams, 0, False)
        got = [t[at].tolist() for t in first]
        assert list(zip(*got)) == [(s, r + g * beams if r >= 0 else r, t, d) for s, r, t, d in want]


@pytest.mark.parametrize("groups,beams,vocab", [(1, 1, 5), (3, 4, 1000), (2, 2, 4099), (40, 8, 32000), (1, 3, 40000)])
def test_a_wait_that_runs_out_fails_its_searches(ck, groups, beams, vocab):
    """Every wait given up at once: no search comes with a candidate, all of them say so, and the next
    call is whole again.  A search of ended and dead beams alone has nothing to wait for."""
    import torch
    rng = np.random.default_rng(vocab)
    rows = groups * beams
    logits = cuda((rng.standard_normal((rows, vocab)) * 65536).astype(np.int64))
    scores, done = cuda(-rng.integers(0, 10 << 16, rows)), cuda(np.zeros(rows, np.uint8))
    exp, plan = cuda(EXP.view(np.int32)), ck.BeamPlan(groups, beams, vocab)
    rc, want = plan.select(logits, scores, done, exp, done_token=vocab - 1)
    assert rc == 0 and (want.done <= 1).all()
    try:
        assert ck.set_beam_wait_limit(1) == 0
        rc, got = plan.select(logits, scores, done, exp, done_token=vocab - 1)
        assert rc == 0
        assert got.scores.tolist() == [MIN] * rows and got.parent.tolist() == [-1] * rows
        assert got.token.tolist() == [vocab - 1] * rows and got.done.tolist() == [ck.BEAM_FAILED] * rows
        rc, ended = plan.select(logits, scores, torch.ones_like(done), exp)
        assert rc == 0 and ended.done.tolist() == [1] * rows
        assert ended.parent.tolist() == [r for g in range(groups) for r in sorted(
            range(g * beams, (g + 1) * beams), key=lambda r: (-int(scores[r]), r))]
    finally:
        ck.set_beam_wait_limit(0)
    rc, again = plan.select(logits, scores, done, exp, done_token=vocab - 1)
    assert rc == 0 and all(torch.equal(a, b) for a, b in zip(want, again))
    rc, after = plan.select(logits, got.scores, got.done, exp)
    assert rc == 0 and after.scores.tolist() == [MIN] * rows and after.done.tolist() == [0] * rows


def near_of(logits, scores, done, beams, done_token):
    """One search over many logits: the plain form with numpy's sums and sorts (distances below 2^63)."""
    found, vocab = [], logits.shape[1]
    for r in range(beams):
        old = int(scores[r])
        if not -2**61 < old < 2**61:
            continue
        if done[r]:
            found.append((-old, r, vocab))
            continue
        d = np.minimum(logits[r].max() - logits[r], 2**62)
        z = int(EXP.astype(np.int64)[np.minimum(d >> 8, 4096)].sum())
        found += [(int(d[i]) + plain_log_sum(z) - old, r, int(i)) for i in np.argsort(d, kind="stable")[:beams]]
    found = sorted(found)[:beams]
    return [(-c, r, done_token if i == vocab else i, int(i == vocab)) for c, r, i in found] + \
        [(MIN, -1, done_token, 0)] * (beams - len(found))


@pytest.mark.parametrize("vocab", [32768, 32769, 50257, 65536, 151936, 2**20 - 1, 2**20])
@pytest.mark.parametrize("beams", [1, 4, 64])
def test_beam_selection_over_large_vocabularies(ck, vocab, beams):
    """More logits than a cluster of eight holds in registers: they are gone through once a pass.  Rows
    of ordinary logits, of many ties, of distances past 32 bits, of one value, and rising ones; the
    largest logits at the ends of the blocks' parts."""
    rng = np.random.default_rng(vocab + beams)
    logits = (rng.standard_normal((max(beams, 4), vocab)) * 3 * 65536).astype(np.int64)
    logits[1] = rng.integers(-3, 3, vocab)
    logits[2] = rng.integers(-2**61, 2**61, vocab)
    logits[3] = np.arange(vocab) if vocab % 2 else 5
    per = -(-vocab // 8)
    logits[0, [vocab - 1, 0, per - 1, min(per, vocab - 1)]] = 2**20
    for shift in range(1 if beams == 64 else 4):
        rows = np.roll(logits, shift, axis=0)[:beams]
        scores, done = -rng.integers(0, 10 << 16, beams), np.zeros(beams, np.uint8)
        if beams == 64:
            scores[5], done[7] = MIN, 1
        rc, got = ck.BeamPlan(1, beams, vocab).select(cuda(rows), cuda(scores), cuda(done), cuda(EXP.view(np.int32)),
                                                      done_token=9)
        assert rc == 0
        assert list(zip(*(t.tolist() for t in got))) == near_of(rows, scores, done, beams, 9)


def single_rows(ck, lens, news, hd, bound, seed=0, **more):
    """A batch whose bounds send it to the kernel of single rows: blocks of the kernel for a few queries
    could not hold the page list of so long a sequence."""
    s = Setup(ck, lens, news, 4, 2, hd, 8, seed=seed, **more)
    s.table = np.concatenate([s.table, np.full((len(lens), bound // 8 + 2), -1, np.int32)], 1)
    s.batch = ck.PagedBatch(cuda(s.table), cuda(np.array(lens, np.int32)), cuda(s.starts), None, s.rows, 320, bound)
    return s


@pytest.mark.parametrize("hd", [4, 16, 32])
def test_single_rows_alone(ck, hd):
    """The kernel for all values on its own, with sequences without rows, without positions, and
    words of 32 and queries of 63 bits."""
    s = single_rows(ck, [400, 33, 8, 0, 2], [320, 5, 0, 1, 4], hd, 300_000, seed=hd, lead=1, tail=2)
    assert ck.paged_attention_work(s.cache, s.batch, 4).numel() == 608 * 300_000 * 8
    wide = s.rng.integers(-2**62, 2**62, (s.rows, 4 * hd))
    q = np.where(np.arange(s.rows)[:, None] % 3 == 0, wide, wide >> 45)
    s.k[s.table[1, 2]] = s.rng.integers(-2**31, 2**31, s.k[0].shape)
    s.v[s.table[1, 2]] = s.rng.integers(-2**31, 2**31, s.k[0].shape)
    s.cache.k.copy_(cuda(s.k))
    s.cache.v.copy_(cuda(s.v))
    import torch
    out = torch.full((s.rows, 4 * hd), 7, dtype=torch.int64, device="cuda")
    rc, _ = ck.paged_attention(s.cache, 1, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 22, out=out)
    assert rc == 0 and s.batch.errors() == [None] * 5
    assert np.array_equal(out.cpu().numpy(), s.attention(1, q, 1 << 22, fill=7))


def test_starts_that_do_not_ascend_stay_within_the_tables(ck):
    """Rows 2 to 8 lie behind the last sequence's end: they have no position, and the last sequence's
    table ends with its length."""
    import torch
    hd = 16
    rng = np.random.default_rng(1)
    cache = ck.PagedCache.empty(4, 1, 1, 8, hd)
    # the table is a view whose last row is followed by other words
    words = cuda(np.array([[0], [1], [2], [3], [3], [3]], np.int32))
    q, k, v = (cuda((rng.standard_normal((9, hd)) * 65536).astype(np.int64)) for _ in range(3))
    batch = ck.PagedBatch(words[:3], cuda(np.array([8, 8, 8], np.int32)), cuda(np.array([0, 9, 1, 2], np.int32)), None,
                          9, 9, 8)
    out = torch.full((9, hd), 5, dtype=torch.int64, device="cuda")
    rc, _ = ck.paged_store(cache, 0, batch, q, k, v, cuda(rope_of(8, 0)), out=out)
    assert rc == 0
    assert (out[2:] == 5).all() and (cache.k[3] == 0).all() and (cache.v[3] == 0).all()
    long = torch.full((3, 300_000 // 8 + 1), 3, dtype=torch.int32, device="cuda")
    long[:, :1] = words[:3]
    many = cuda(np.concatenate([[0, 900, 1], np.arange(2, 321)]).astype(np.int32))
    wide = ck.PagedBatch(long[:1].expand(321, -1).contiguous(), cuda(np.full(321, 8, np.int32)), many, None, 900, 320, 300_000)
    out = torch.full((900, hd), 5, dtype=torch.int64, device="cuda")
    rows = cuda((rng.standard_normal((900, hd)) * 65536).astype(np.int64))
    assert ck.paged_attention_work(cache, wide, 1).numel() == 608 * 300_000 * 8      # the kernel of single rows
    rc, _ = ck.paged_attention(cache, 0, wide, rows, cuda(EXP.view(np.int32)), 1 << 22, out=out)
    assert rc == 0
    assert (out[320:] == 5).all()
    assert wide.errors()[2:] == [None] * 319


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("heads,kv,hd,rot", [(15, 3, 64, 48), (5, 5, 128, 128), (33, 1, 32, 0)])
def test_store_of_rows_that_fill_the_gpu(ck, heads, kv, hd, rot, half):
    """A block a row whose threads take several units, the last ones not all of them: words that do not
    fit, rows of no sequence, and rows without a position among them."""
    import torch
    lens, news = [411, 90, 300, 3], [411, 0, 290, 6]
    s = Setup(ck, lens, news, heads, kv, hd, 16, seed=heads, lead=1, tail=2)
    units = (heads + 2 * kv) * hd // 4
    assert s.rows >= 4 * torch.cuda.get_device_properties(0).multi_processor_count and 256 < units and units % 256
    qkv = (s.rng.standard_normal((s.rows, (heads + 2 * kv) * hd)) * 65536).astype(np.int64)
    parts = np.split(qkv, [heads * hd, (heads + kv) * hd], axis=1)
    parts[1][7, kv * hd - 1], parts[2][500, kv * hd - 2], parts[0][3, 5] = 2**31, -2**40, 2**62
    qkv = np.concatenate(parts, axis=1)
    rope = rope_of(max(lens), rot)
    out = torch.zeros(s.rows, heads * hd, dtype=torch.int64, device="cuda")
    dev = cuda(qkv).split((heads * hd, kv * hd, kv * hd), -1)
    rc, q = ck.paged_store(s.cache, 1, s.batch, *dev, cuda(rope), half=half, out=out)
    assert rc == 0
    qo, pk, pv, status = plain_store(s, 1, *parts, rope, half)
    assert np.array_equal(q.cpu().numpy(), qo)
    assert np.array_equal(s.cache.k.cpu().numpy(), pk) and np.array_equal(s.cache.v.cpu().numpy(), pv)
    assert status[0] is not None and status[2] is not None and s.batch.errors() == status


def fork_beside(lens, table, parent, grow, pages, page, shared):
    """The plain fork where `shared` pages are another sequence's: as if one more output row had each
    of them whole."""
    stride = max(table.shape[1], len(shared))
    wide = np.full((len(lens) + 1, stride), -1)
    wide[:-1, :table.shape[1]], wide[-1, :len(shared)] = table, shared
    out, out_lens, status, copies = plain_fork(list(lens) + [len(shared) * page], wide, list(parent) + [len(lens)],
                                               list(grow) + [0], pages, page)
    return out[:-1, :table.shape[1]], out_lens[:-1], status[:-1], copies


@pytest.mark.parametrize("page,hd,rows,n", [(8, 16, 3, 21), (16, 4, 1, 5), (8, 8, 40, 63), (32, 64, 2, 64)])
def test_a_kept_prompt_forked_again_and_again(ck, page, hd, rows, n):
    """Each fork extends every row by a position and writes it.  The prompt's pages and those of the
    rows of the forks before are shared: nothing that a live sequence wrote is written again."""
    rng = np.random.default_rng(n)
    stride = -(-(n + 1) // page) + 1
    pages = 4 * rows * stride
    k, v = pools(rng, pages, 2, 1, page, hd)
    cache = ck.PagedCache(cuda(k), cuda(v))
    plan = ck.PagePlan(cache, rows, stride)
    prompt = np.full((1, stride), -1, np.int32)
    prompt[0, :-(-n // page)] = rng.permutation(pages)[:-(-n // page)]
    live, words = [], {}
    for turn in range(3):
        shared = sorted({int(w) for t in [prompt] + live for w in t.flatten() if w >= 0})
        held = np.where(np.isin(np.arange(pages), shared), ck.PAGE_SHARED, 0).astype(np.uint8)
        parent, grow = np.zeros(rows, np.int32), np.ones(rows, np.int32)
        rc, got = plan.fork(cuda(parent), cuda(np.array([n], np.int32)), cuda(prompt), cuda(grow), held=cuda(held))
        assert rc == 0
        want, want_lens, status, copies = fork_beside([n], prompt, parent, grow, pages, page, shared)
        assert got.status.tolist() == status == [0] * rows and got.lens.tolist() == want_lens
        table = got.table.cpu().numpy()
        assert np.array_equal(table, want) and len(copies) == (rows if n % page else 0)
        for src, dst, m in copies:
            k[dst, :, :, :m], v[dst, :, :, :m] = k[src, :, :, :m], v[src, :, :, :m]
        assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
        for r in range(rows):                         # position n of the row
            at = int(table[r, n // page]), n % page
            assert at not in words
            words[at] = 1000 * turn + r
            k[at[0], :, :, at[1]] = words[at]
        cache.k.copy_(cuda(k))
        live.append(table)
    pool = cache.k.cpu().numpy()
    for at, word in words.items():
        assert (pool[at[0], :, :, at[1]] == word).all()


def test_marks_of_held_pages(ck):
    """A reserved page stays with its first row, a shared one (and one marked with both) with none; a
    row whose copy finds no page is empty, and the rows behind it too."""
    rng = np.random.default_rng(11)
    page, pages = 8, 12
    k, v = pools(rng, pages, 1, 2, page, 8)
    table, lens = np.array([[3, 5, -1, -1], [9, -1, -1, -1]]), [13, 4]
    for mark, full in ((1, False), (2, False), (3, False), (2, True)):
        cache = ck.PagedCache(cuda(k), cuda(v))
        held = np.zeros(pages, np.uint8)
        held[5], held[9] = mark, 1
        if full:
            held[[w for w in range(pages) if w not in (3, 5, 9, 11)]] = 1
        rc, got = ck.PagePlan(cache, 3, 4).fork(cuda(np.array([0, 0, 1], np.int32)), cuda(np.array(lens, np.int32)),
                                                cuda(table.astype(np.int32)), cuda(np.array([1, 1, 1], np.int32)),
                                                held=cuda(held))
        assert rc == 0
        if full:
            assert got.status.tolist() == [0, 4, 4] and got.lens.tolist() == [14, 0, 0]
            assert got.table.tolist() == [[3, 11, -1, -1], [-1] * 4, [-1] * 4]
        else:
            assert got.status.tolist() == [0] * 3 and got.lens.tolist() == [14, 14, 5]
            first = [3, 5, -1, -1] if mark == 1 else [3, 0, -1, -1]
            assert got.table.tolist() == [first, [3, 0 if mark == 1 else 1, -1, -1], [9, -1, -1, -1]]
        pool = cache.k.cpu().numpy()
        for row in got.table.tolist():
            if row[1] >= 0:
                assert np.array_equal(pool[row[1], :, :, :5], k[5, :, :, :5])
        assert np.array_equal(pool[5], k[5])


@pytest.mark.parametrize("lens,news,heads,kv,hd,page,bound", [
    ([700], [300], 32, 8, 32, 16, 60_000),                           # groups of queries of one sequence
    ([300, 0, 41, 555], [160, 3, 0, 161], 8, 8, 4, 8, 100_000),      # of several, ragged
    ([int(n) for n in np.arange(200) * 7 % 45], [1] * 200, 4, 4, 16, 256, 500_000),  # whole sequences
])
def test_attention_in_launches_that_share_the_scratch(ck, lens, news, heads, kv, hd, page, bound):
    """Bounds so large that the scores of all queries at once would pass two gigabytes."""
    import torch
    s = Setup(ck, lens, news, heads, kv, hd, page, seed=hd, lead=2, tail=1)
    s.table = np.concatenate([s.table, np.full((len(lens), bound // page + 2), -1, np.int32)], 1)
    s.batch = ck.PagedBatch(cuda(s.table), cuda(np.array(lens, np.int32)), cuda(s.starts), None, s.rows, max(news), bound)
    queries = max(news) * heads // kv
    assert 8 * bound * kv * len(lens) * (queries if queries > 1 else 1) > 2**31
    assert 2**30 < ck.paged_attention_work(s.cache, s.batch, heads).numel() <= 2**31
    q = (s.rng.standard_normal((s.rows, heads * hd)) * 65536).astype(np.int64)
    out = torch.full((s.rows, heads * hd), 7, dtype=torch.int64, device="cuda")
    rc, _ = ck.paged_attention(s.cache, 1, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 22, out=out)
    assert rc == 0 and s.batch.errors() == [None] * len(lens)
    assert np.array_equal(out.cpu().numpy(), s.attention(1, q, 1 << 22, fill=7))


def test_numbers_that_are_no_u32_are_refused(ck):
    s = Setup(ck, [20], [2], 2, 2, 16, 8)
    b, exp = s.batch, cuda(EXP.view(np.int32))
    q = cuda(np.zeros((2, 32), np.int64))
    for rows, max_new, max_len in ((2**32 + 2, 2, 20), (2, 2**32 + 2, 20), (2, 2, 2**32 + 20), (2, 2, -1)):
        with pytest.raises(ValueError):
            ck.PagedBatch(b.table, b.lens, b.starts, b.status, rows, max_new, max_len)
    for layer, inv in ((2**32, 1), (-1, 1), (0, 2**32), (0, -1)):
        with pytest.raises(ValueError):
            ck.paged_attention(s.cache, layer, b, q, exp, inv)
    with pytest.raises(ValueError):
        ck.paged_store(s.cache, 2**32, b, q, q, q, cuda(rope_of(20, 16)))
    plan = ck.BeamPlan(1, 1, 9)
    with pytest.raises(ValueError):
        plan.select(cuda(np.zeros((1, 9), np.int64)), cuda(np.zeros(1, np.int64)), cuda(np.zeros(1, np.uint8)), exp,
                    done_token=2**32)


def test_what_plans_and_caches_allocated_stays_in_use_on_another_current_stream(ck):
    """The current stream is busy when the calls are enqueued; then the plan, the cache and the batch
    (its status words too) are dropped and their memory is asked for again on the stream that they
    were made on, before the kernels run."""
    import torch
    rng = np.random.default_rng(4)
    logits, scores = rng.integers(0, 2**20, (4, 900)), np.zeros(4, np.int64)
    dev = cuda(logits), cuda(scores), cuda(np.zeros(4, np.uint8)), cuda(EXP.view(np.int32))
    parent, lens, grow = cuda(np.zeros(4, np.int32)), cuda(np.array([9], np.int32)), cuda(np.ones(4, np.int32))
    table, starts = cuda(np.array([[5, 2, -1]], np.int32)), cuda(np.array([0, 1], np.int32))
    q = cuda((rng.standard_normal((1, 16)) * 65536).astype(np.int64))
    side = torch.cuda.Stream()

    def calls():
        plan, cache = ck.BeamPlan(1, 4, 900), ck.PagedCache.empty(12, 1, 1, 8, 16)
        move, batch = ck.PagePlan(cache, 4, 3), ck.PagedBatch(table, lens, starts, None, 1, 1, 9)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
            rc, beams = plan.select(*dev)
            assert rc == 0
            rc, fork = move.fork(parent, lens, table, grow)
            assert rc == 0
            rc, _ = ck.paged_store(cache, 0, batch, q, q, q, cuda(rope_of(9, 0)))
            assert rc == 0
            rc, out = ck.paged_attention(cache, 0, batch, q, dev[3], 1 << 22)
            assert rc == 0
        return beams, fork, out

    for t in (torch.int32, torch.int64, torch.uint8):  # (every kernel below is loaded before the stream is busy)
        torch.full((3,), 3, dtype=t, device="cuda")
    calls()
    torch.cuda.synchronize()
    beams, fork, out = calls()
    sizes = [1 << n for n in range(8, 18)]
    other = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(100)]
    torch.cuda.synchronize()
    assert list(zip(*(t.tolist() for t in beams))) == plain_beam(logits, scores, np.zeros(4), 1, 4, 0, False)
    assert fork.table.tolist() == [[5, 2, -1], [5, 0, -1], [5, 1, -1], [5, 3, -1]] and fork.status.tolist() == [0] * 4
    # position 8 of nine: the positions before it hold zeros, so the value is a part of its word
    k = np.zeros((9, 16), np.int64)
    k[8] = q.cpu().numpy()
    assert np.array_equal(out.cpu().numpy()[0], plain_attention(k[8], k, k, 1 << 22))
    assert all((t == 3).all() for t in other)


def test_a_pool_without_heads_or_elements_is_refused(ck):
    s = Setup(ck, [20], [2], 2, 2, 16, 8)
    q, exp = cuda(np.zeros((2, 32), np.int64)), cuda(EXP.view(np.int32))
    for shape in ((3, 1, 2, 8, 0), (3, 1, 0, 8, 16)):
        cache = ck.PagedCache.empty(*shape)
        with pytest.raises(ValueError):
            ck.paged_attention(cache, 0, s.batch, q, exp, 1)
        with pytest.raises(ValueError):
            ck.paged_store(cache, 0, s.batch, q, q, q, cuda(rope_of(20, 16)))


def test_sequences_longer_than_their_tables_are_skipped(ck):
    """Lengths within max_len that the tables have no entries for, in all three kernels and the store."""
    import torch
    for lens, news, heads, kv, hd, page in (([40, 33], [2, 2], 4, 2, 32, 8), ([900, 700], [70, 129], 32, 8, 64, 16)):
        s = Setup(ck, lens, news, heads, kv, hd, page, seed=2, max_len=lens[0] + 500)
        at = s.table.shape[1] * page
        s.batch.lens.copy_(cuda(np.array([at + 1, lens[1]], np.int32)))
        assert on_tiles(ck, s) == (hd == 64)
        q = (s.rng.standard_normal((s.rows, heads * hd)) * 65536).astype(np.int64)
        want = s.attention(1, q, 1 << 21)
        out = torch.full((s.rows, heads * hd), 5, dtype=torch.int64, device="cuda")
        rc, _ = ck.paged_attention(s.cache, 1, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 21, out=out)
        assert rc == 0 and s.batch.errors() == [(0, 1, 1, 0), None]
        got = out.cpu().numpy()
        assert (got[:news[0]] == 5).all() and np.array_equal(got[news[0]:], want[news[0]:])
        k, before = cuda(q[:, :kv * hd]), s.cache.k.clone()
        s.batch.status.fill_(-1)
        out.fill_(5)
        rc, _ = ck.paged_store(s.cache, 0, s.batch, cuda(q), k, k, cuda(rope_of(at + 1, 0)), out=out)
        assert rc == 0 and s.batch.errors() == [(0, 0, 1, 0), None]
        assert (out[:news[0]] == 5).all() and torch.equal(out[news[0]:], cuda(q)[news[0]:])
        mine = [int(p) for p in s.table[0] if p >= 0]
        assert torch.equal(s.cache.k[mine], before[mine])
    s = single_rows(ck, [400, 30], [317, 3], 16, 300_000)
    s.batch = ck.PagedBatch(s.batch.table[:, :300_000 // 8].contiguous(), cuda(np.array([300_000, 30], np.int32)), s.batch.starts,
                            None, s.rows, 320, 300_001)
    s.batch.lens[0] = 300_001
    q = (s.rng.standard_normal((s.rows, 64)) * 65536).astype(np.int64)
    out = torch.full((s.rows, 64), 5, dtype=torch.int64, device="cuda")
    assert ck.paged_attention_work(s.cache, s.batch, 4).numel() >= 608 * 300_000 * 8
    rc, _ = ck.paged_attention(s.cache, 0, s.batch, cuda(q), cuda(EXP.view(np.int32)), 1 << 22, out=out)
    assert rc == 0 and s.batch.errors() == [(0, 0, 1, 0), None]
    assert (out[:317] == 5).all() and np.array_equal(out[317:].cpu().numpy(), s.attention(0, q, 1 << 22)[317:])


@pytest.mark.parametrize("groups,beams,vocab", [(1, 64, 1), (3, 64, 2), (1000, 64, 3), (65536, 1, 2)])
def test_beams_with_hardly_a_vocabulary(ck, groups, beams, vocab):
    rng = np.random.default_rng(beams)
    rows = groups * beams
    logits = rng.integers(-2**17, 2**17, (rows, vocab))
    scores, done = -rng.integers(0, 5 << 16, rows), (rng.random(rows) < 0.2).astype(np.uint8)
    rc, got = ck.BeamPlan(groups, beams, vocab).select(cuda(logits), cuda(scores), cuda(done), cuda(EXP.view(np.int32)))
    assert rc == 0
    got = list(zip(*(t.tolist() for t in got)))
    for g in sorted({0, 1 % groups, groups // 3, groups - 1}):
        at = slice(g * beams, (g + 1) * beams)
        want = plain_beam(logits[at], scores[at], done[at], 1, beams, 0, False)
        assert got[at] == [(s, r + g * beams if r >= 0 else r, t, d) for s, r, t, d in want]
