"""A model's layers over a cache in pages, and searches with it: logits against the CPU oracle's
and beam search against one that recomputes every hypothesis, bit for bit."""
import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu

MIN = -2**63


@pytest.fixture(scope="module")
def ck():
    import torch
    import fixed_point_int8_gb300 as ck
    from fixed_point_int8_gb300 import build
    build.build()
    torch.cuda.init()
    return ck


class Both:
    def __init__(self, ck, spec):
        self.spec = spec
        art = synth.build_artifact(spec)
        self.orc = oracle.Model(art)
        rc, self.gpu = ck.Model.load(art)
        assert rc == 0

    def logits(self, ids):
        """The oracle's logits behind the tokens."""
        rc, state = self.orc.init_state(np.array(ids, np.uint32), 1)
        assert rc == 0
        assert self.orc.turn(state, len(ids))[0] == 0
        at = self.orc.layout(len(ids), 1)["logits"]
        return state[at:at + 8 * self.spec.vocab].view("<i8").copy()

    def cache(self, ck, pages, page):
        return ck.PagedCache.empty(pages, self.spec.layers, self.spec.kv_heads, page, self.spec.dim // self.spec.heads)


@pytest.fixture(scope="module")
def gqa(ck):
    return Both(ck, synth.GQA)


def i32(a):
    import torch
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def test_tables_of_the_model(ck, gqa):
    assert np.array_equal(gqa.gpu.exp_table().cpu().numpy().view(np.uint32), synth.exp_table())


@pytest.mark.parametrize("page,sizes", [(8, (5, 1, 17)), (16, (40, 33)), (32, (2,))])
def test_prompts_in_chunks_then_single_tokens(ck, gqa, page, sizes):
    """Ragged chunks of several prompts, then one token a sequence: every pass's logits are the
    oracle's for the tokens so far."""
    spec, seqs = gqa.spec, len(sizes)
    ids = [[int(t) for t in synth.prompt_ids(spec, n + 6, run=i)] for i, n in enumerate(sizes)]
    cache = gqa.cache(ck, 40, page)
    plan = ck.PagePlan(cache, seqs, 128 // page)
    table, lens = i32(np.full((seqs, 128 // page), -1)), i32([0] * seqs)
    first = [(n + 1) // 2 for n in sizes]
    steps = [first, [n - f for n, f in zip(sizes, first)]] + [[1] * seqs] * 4
    done = [0] * seqs
    for news in steps:
        rc, got = plan.fork(i32(range(seqs)), lens, table, i32(news))
        assert rc == 0 and got.status.tolist() == [0] * seqs
        table, lens = got.table, got.lens
        tokens = [t for i, n in enumerate(news) for t in ids[i][done[i]:done[i] + n]]
        done = [d + n for d, n in zip(done, news)]
        if not tokens:
            continue
        batch = ck.PagedBatch(table, lens, i32(np.cumsum([0] + news)), None, len(tokens), max(news), max(done))
        rc, logits = gqa.gpu.turn_paged(cache, batch, i32(tokens))
        assert rc == 0 and batch.errors() == [None] * seqs
        for i, n in enumerate(news):
            if n:
                assert np.array_equal(logits[i].cpu().numpy(), gqa.logits(ids[i][:done[i]])), (i, done[i])


def test_a_larger_model_over_pages_agrees_with_the_batched_turn(ck):
    """Head size 64 and a chunk that goes to the tensor-core attention: the logits of the last
    prompt position are those of a run's own state after ck_turn."""
    spec = synth.ModelSpec("hd64", 512, 352, 2, 8, 2, 512, 512, tied=False, seed=0x5EED0077)
    both, n = Both(ck, spec), 400
    ids = [int(t) for t in synth.prompt_ids(spec, n)]
    state = both.gpu.new_state(n, 1)
    assert both.gpu.init_state(state, ids, 1) == 0
    assert both.gpu.turn(state, n)[0] == 0
    rc, want = both.gpu.logits(state)
    assert rc == 0
    cache = both.cache(ck, 28, 16)
    batch = ck.PagedBatch(i32([list(range(27, 2, -1))]), i32([n]), i32([0, n]), None, n, n, n)
    assert ck.paged_attention_work(cache, batch, 8).numel() > 1 << 20   # the tiles
    rc, logits = both.gpu.turn_paged(cache, batch, i32(ids))
    assert rc == 0 and batch.errors() == [None]
    assert np.array_equal(logits[0].cpu().numpy(), want)


def test_failures_are_each_sequences_own(ck, gqa):
    """A token outside the vocabulary, a page outside the pool, a sequence without new rows and a
    row of no sequence: the others' logits are the oracle's."""
    import torch
    ids = [int(t) for t in synth.prompt_ids(gqa.spec, 9)]
    cache = gqa.cache(ck, 8, 8)
    tokens = [ids[0], 512] + ids[:9] + [ids[0]] + [-1, 7]
    table = i32([[0, -1], [1, 2], [9, -1], [3, -1]])
    batch = ck.PagedBatch(table, i32([2, 9, 1, 4]), i32([0, 2, 11, 12, 12]), None, 14, 9, 16)
    logits = torch.full((4, 512), 5, dtype=torch.int64, device="cuda")
    rc, _ = gqa.gpu.turn_paged(cache, batch, i32(tokens), logits=logits)
    assert rc == 0
    assert batch.errors() == [(1, 0, 3, 0), None, (0, 0, 2, 0), None]
    assert np.array_equal(logits[1].cpu().numpy(), gqa.logits(ids))
    assert (logits[3] == 5).all()


def plain_search(both, prompt, beams, steps, step):
    """Beam search that runs the oracle over every hypothesis from its first token; `step` is the
    selection over plain logits."""
    hyps = [(list(prompt), 0, False)] + [(list(prompt), MIN, False)] * (beams - 1)
    for _ in range(steps):
        rows = [both.logits(h[0]) if h[1] != MIN and not h[2] else np.zeros(both.spec.vocab, np.int64) for h in hyps]
        got = step(np.array(rows), [h[1] for h in hyps], [int(h[2]) for h in hyps])
        hyps = [(hyps[r][0] + [t], s, bool(d)) if r >= 0 else ([], MIN, False) for s, r, t, d in got]
    return hyps


@pytest.mark.parametrize("page,beams,captured", [(8, 4, False), (16, 3, False), (8, 4, True)])
def test_beam_search_over_pages(ck, gqa, page, beams, captured):
    """Selection, reordering of the pages, stores and attention together, for two searches at once;
    the captured form replays one step's kernels."""
    import torch
    from test_gpu_paged import plain_beam
    spec, groups, steps = gqa.spec, 2, 6
    prompts = [[int(t) for t in synth.prompt_ids(spec, n, run=i)] for i, n in enumerate((7, 16))]
    rows, stride = groups * beams, 8
    cache = gqa.cache(ck, 30, page)
    plan, select = ck.PagePlan(cache, rows, stride), ck.BeamPlan(groups, beams, spec.vocab)
    exp = gqa.gpu.exp_table()
    # the prompts, one row each
    rc, got = plan.fork(i32([0, 1]), i32([0, 0]), i32(np.full((2, stride), -1)), i32([7, 16]))
    assert rc == 0
    batch = ck.PagedBatch(got.table, got.lens, i32([0, 7, 23]), None, 23, 16, 16)
    rc, first = gqa.gpu.turn_paged(cache, batch, i32(prompts[0] + prompts[1]))
    assert rc == 0 and batch.errors() == [None, None]
    # a search starts with one live beam; the others share its pages from the first selection on
    of = torch.arange(rows, device="cuda") // beams
    logits, table, lens = first[of].contiguous(), got.table[of].contiguous(), got.lens[of].contiguous()
    scores = torch.where(torch.arange(rows, device="cuda") % beams == 0, 0, MIN)
    done = torch.zeros(rows, dtype=torch.uint8, device="cuda")
    ones, starts = i32([1] * rows), i32(range(rows + 1))
    status = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    work = None
    history = []

    def step(logits, scores, done, table, lens):
        nonlocal work
        rc, b = select.select(logits, scores, done, exp, stop_tokens=True, done_token=2)
        assert rc == 0
        rc, f = plan.fork(b.parent, lens, table, ones)
        assert rc == 0
        batch = ck.PagedBatch(f.table, f.lens, starts, status, rows, 1, 40)
        if work is None:
            work = gqa.gpu.turn_paged_work(cache, batch)
        rc, out = gqa.gpu.turn_paged(cache, batch, b.token, work=work)
        assert rc == 0
        return b, f, out

    if captured:
        static = [t.clone() for t in (logits, scores, done, table, lens)]
        pools = cache.k.clone(), cache.v.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(*static)                          # what is set up once is set up before the capture
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b, f, out = step(*static)
            for to, new in zip(static, (out, b.scores, b.done, f.table, f.lens)):
                to.copy_(new)
        cache.k.copy_(pools[0])
        cache.v.copy_(pools[1])
        for to, new in zip(static, (logits, scores, done, table, lens)):
            to.copy_(new)
        for _ in range(steps):
            graph.replay()
            history.append((b.parent.tolist(), b.token.tolist()))
            assert f.status.tolist() == [0] * rows
        final_scores, final_done = static[1].tolist(), static[2].tolist()
    else:
        for _ in range(steps):
            b, f, logits = step(logits, scores, done, table, lens)
            scores, done, table, lens = b.scores, b.done, f.table, f.lens
            history.append((b.parent.tolist(), b.token.tolist()))
            assert f.status.tolist() == [0] * rows
        final_scores, final_done = scores.tolist(), done.tolist()
    assert status.tolist() == [-1] * rows
    for g in range(groups):
        want = plain_search(gqa, prompts[g], beams, steps,
                            lambda lo, sc, dn: plain_beam(lo, sc, dn, 1, beams, 2, True))
        for j in range(beams):
            r, tokens = g * beams + j, []
            assert final_scores[r] == want[j][1] and bool(final_done[r]) == want[j][2]
            for parent, token in reversed(history):
                tokens.append(token[r])
                r = parent[r]
            assert prompts[g] + tokens[::-1] == want[j][0]


def test_a_paged_turn_on_another_stream_and_two_at_once(ck, gqa):
    """Two sequences' passes at the same time on streams of their own, with scratch of their own."""
    import torch
    ids = [[int(t) for t in synth.prompt_ids(gqa.spec, 30, run=i)] for i in range(2)]
    want = [gqa.logits(i) for i in ids]
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    jobs = []
    for i in range(2):
        cache = gqa.cache(ck, 6, 8)
        jobs.append((cache, ck.PagedBatch(i32([[3, 1, 0, 5]]), i32([30]), i32([0, 30]), None, 30, 30, 30), i32(ids[i])))
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for (cache, batch, tokens), stream in zip(jobs, streams):
            rc, logits = gqa.gpu.turn_paged(cache, batch, tokens, stream=stream)
            assert rc == 0
            outs.append(logits)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert np.array_equal(o[0].cpu().numpy(), w)


@pytest.mark.parametrize("change", [dict(layers=4), dict(kv_heads=2), dict(head_dim=16)])
def test_a_cache_of_another_model_is_refused(ck, gqa, change):
    shape = dict(layers=5, kv_heads=4, head_dim=8)
    shape.update(change)
    cache = ck.PagedCache.empty(4, shape["layers"], shape["kv_heads"], 8, shape["head_dim"])
    batch = ck.PagedBatch(i32([[0, 1]]), i32([3]), i32([0, 3]), None, 3, 3, 8)
    with pytest.raises(ck.CkError):
        gqa.gpu.turn_paged_work(cache, batch)
    long = ck.PagedBatch(i32([[0, 1]]), i32([3]), i32([0, 3]), None, 3, 3, 513)  # past the context
    with pytest.raises(ck.CkError):
        gqa.gpu.turn_paged_work(gqa.cache(ck, 4, 8), long)


def test_more_sequences_than_rows(ck, gqa):
    """Seventy sequences of which two have a new token, in a pass on another current stream: the
    classifier runs for all of them, in more columns than the layers."""
    import torch
    ids = [[int(t) for t in synth.prompt_ids(gqa.spec, n, run=n)] for n in (6, 9)]
    cache = gqa.cache(ck, 70, 16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        first = ck.PagedBatch(i32([[5], [60]]), i32([5, 8]), i32([0, 5, 13]), None, 13, 8, 8)
        rc, _ = gqa.gpu.turn_paged(cache, first, i32(ids[0][:5] + ids[1][:8]))
        assert rc == 0
        lens, starts, table = [0] * 70, [0] * 71, [[-1]] * 70
        lens[3], lens[69], table[3], table[69] = 6, 9, [5], [60]
        starts[4:70], starts[70] = [1] * 66, 2
        batch = ck.PagedBatch(i32(table), i32(lens), i32(starts), None, 2, 1, 16)
        logits = torch.full((70, 512), 7, dtype=torch.int64, device="cuda")
        rc, _ = gqa.gpu.turn_paged(cache, batch, i32([ids[0][5], ids[1][8]]), logits=logits)
        assert rc == 0 and batch.errors() == [None] * 70 and first.errors() == [None] * 2
    torch.cuda.synchronize()
    for at, run in ((3, ids[0]), (69, ids[1])):
        assert np.array_equal(logits[at].cpu().numpy(), gqa.logits(run))
    keep = [i for i in range(70) if i not in (3, 69)]
    assert (logits[keep] == 7).all()
