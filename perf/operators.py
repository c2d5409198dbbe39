"""The operators of the paged key/value cache and of beam search, as they are measured: their
cases, inputs and plain forms in elementary torch operations on 64-bit integers.

Formats are the library's: queries, keys, values before their store, logits and scores are
int64 with 16 fraction bits, cached words int32 with 16, rotary entries int32 with 24, the
exponential table 4,097 entries with 30.  A pool is int32 [pages][layers][kv heads][page][head];
a table row lists a sequence's pages in order, -1 where there is none."""
import math

import torch

own = False

MIN = -2**63
DEAD = -2**61          # a beam whose score is at or below this is dead
NO_ROW = -1            # the parent of an output row that holds nothing
LN2 = 744261118        # ln 2 with 30 fraction bits


def listed():
    return [
        # one run of the 1B shape late in its 8K context: a single new token, all of the cache read
        {"name": "attend_1b_8191", "op": "attend", "seqs": 1, "new": 1, "len_min": 8191, "len": 8191,
         "heads": 32, "kv_heads": 32, "head": 64, "page": 64, "layers": 1},
        # 64 runs of the 1B shape, each at a position of its own: one new token a run
        {"name": "attend_1b_64runs", "op": "attend", "seqs": 64, "new": 1, "len_min": 65, "len": 191,
         "heads": 32, "kv_heads": 32, "head": 64, "page": 16, "layers": 1},
        # chunks of two prompts of the 7B shape, ragged in new tokens and in length
        {"name": "attend_7b_chunk", "op": "attend", "seqs": 2, "new": 201, "len_min": 777, "len": 2047,
         "heads": 32, "kv_heads": 32, "head": 128, "page": 32, "layers": 1},
        # the last chunk of a long prompt of the 1B shape
        {"name": "attend_1b_chunk_7936", "op": "attend", "seqs": 1, "new": 256, "len_min": 7936, "len": 7936,
         "heads": 32, "kv_heads": 32, "head": 64, "page": 64, "layers": 1},
        # a decode step's queries, keys and values of one run of the 7B shape
        {"name": "store_7b_1", "op": "store", "seqs": 1, "new": 1, "len_min": 133, "len": 133, "heads": 32,
         "kv_heads": 32, "head": 128, "page": 16, "layers": 1, "rot": 128, "half": False},
        # prompts of eight runs of the 1B shape, half layout on half of each head
        {"name": "store_1b_2040", "op": "store", "seqs": 8, "new": 255, "len_min": 255, "len": 1021, "heads": 32,
         "kv_heads": 32, "head": 64, "page": 16, "layers": 1, "rot": 32, "half": True},
        # one search of four beams on a small grouped-head model
        {"name": "fork_gqa_1x4", "op": "fork", "groups": 1, "beams": 4, "len_min": 45, "len": 45, "kv_heads": 4,
         "head": 8, "page": 16, "layers": 5},
        # 32 searches of four beams of the 1B shape
        {"name": "fork_1b_32x4", "op": "fork", "groups": 32, "beams": 4, "len_min": 65, "len": 127,
         "kv_heads": 32, "head": 64, "page": 16, "layers": 22},
        # a small pool and a large one packed after runs have left holes
        {"name": "compact_gqa_8", "op": "compact", "groups": 2, "beams": 4, "len_min": 30, "len": 90,
         "kv_heads": 4, "head": 8, "page": 16, "layers": 5},
        {"name": "compact_1b_64", "op": "compact", "groups": 16, "beams": 4, "len_min": 65, "len": 127,
         "kv_heads": 32, "head": 64, "page": 16, "layers": 22},
        # one search of four beams over the vocabulary, and 64 searches of eight
        {"name": "beam_1x4", "op": "beam", "groups": 1, "beams": 4, "vocab": 32000},
        {"name": "beam_64x8", "op": "beam", "groups": 64, "beams": 8, "vocab": 32000},
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["attend", "attend", "store", "fork", "compact", "beam"])
    if op == "beam":
        return {"op": op, "groups": log(1, 64), "beams": rng.randint(1, 8), "vocab": log(7, 32000)}
    c = {"op": op, "head": rng.choice([4, 8, 16, 32, 64, 128]), "page": rng.choice([8, 16, 32, 64]), "layers": 1}
    c["kv_heads"] = rng.choice([1, 2, 4, 8, 32 if c["head"] <= 64 else 8])
    if op in ("fork", "compact"):
        longest = log(17, 127)
        c.update(groups=log(1, 16), beams=rng.randint(1, 8), len=longest, len_min=rng.randint(1, longest),
                 layers=rng.choice([1, 2, 5, 22]))
        return c
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4] if c["kv_heads"] <= 8 else [1])
    if op == "store":
        c.update(seqs=log(1, 8), new=log(1, 255))
        c["rot"] = rng.choice([c["head"], c["head"] // 2])
        c["half"] = rng.choice([False, True])
        c["len"] = rng.randint(c["new"], c["new"] + 766)
    elif rng.random() < 0.5:
        c.update(seqs=log(1, 64), new=1)
        c["len"] = log(1, 8191 // c["seqs"] + 64)
    else:
        c.update(seqs=rng.randint(1, 2), new=log(2, 201))
        c["len"] = c["new"] + rng.randint(0, 1700)
    c["len_min"] = rng.randint((c["len"] + 1) // 2, c["len"])
    return c


# ------------------------------------------------------------------ sizes

def _lens(c):
    """Positions of each row's sequence, new ones included: from the least to the most."""
    n = c["seqs"] if "seqs" in c else c["groups"] * c["beams"]
    return [c["len"] - (c["len"] - c["len_min"]) * i // max(1, n - 1) for i in range(n)]


def _news(c):
    """New tokens of each sequence: the first has c["new"], the others less."""
    return [max(1, min(n, c["new"] - (c["new"] * i) // (2 * c["seqs"]))) for i, n in enumerate(_lens(c))]


def _group_lens(c):
    """Beams of one search are at the same position."""
    g = c["groups"]
    return [c["len"] - (c["len"] - c["len_min"]) * (i // c["beams"]) // max(1, g - 1) for i in range(g * c["beams"])]


def _row_pages(c):
    """Pages of each row of a search: the first half of the full ones are its group's own."""
    lens = _group_lens(c)
    return lens, [-(-n // c["page"]) for n in lens], [n // c["page"] // 2 for n in lens]


def _pages_held(c):
    """Pages in use, anywhere in a pool half as large again and some more."""
    lens, pages, shared = _row_pages(c)
    held = sum(p - h for p, h in zip(pages, shared)) + sum(shared[::c["beams"]])
    return held, held + held // 2 + 2 * len(lens)


def work(case):
    c = case
    if c["op"] == "beam":
        rows = c["groups"] * c["beams"]
        n = rows * c["vocab"]
        return {"bytes": 8 * n + 4 * 4097 + 26 * rows, "flops": 4 * n}
    hd, kv = c["head"], c["kv_heads"]
    if c["op"] in ("fork", "compact"):
        lens, pages, shared = _row_pages(c)
        per = 8 * c["layers"] * kv * hd      # K and V bytes of a position
        table = 8 * sum(pages)
        if c["op"] == "compact":              # the pages beyond the packed range, as many as chance puts there
            held, total = _pages_held(c)
            return {"bytes": table + 2 * per * c["page"] * (held * (total - held) // total), "flops": held}
        # rows whose part-filled page stays with an earlier child of the same parent, by expectation
        b = c["beams"]
        share = [math.sqrt((i + 1) / b) - math.sqrt(i / b) for i in range(b)]
        copied = 1 - sum(1 - (1 - p)**b for p in share) / b
        part = sum(n % c["page"] for n in lens)
        return {"bytes": table + 2 * per * int(part * copied), "flops": sum(pages)}
    news, lens = _news(c), _lens(c)
    rows = sum(news)
    if c["op"] == "store":
        return {"bytes": rows * (16 * c["heads"] * hd + 24 * kv * hd + 4 * c["rot"]),
                "flops": rows * (c["heads"] + kv) * c["rot"] * 3}
    pairs = sum(k * n - k * (k - 1) // 2 for k, n in zip(news, lens))
    return {"bytes": 16 * rows * c["heads"] * hd + 8 * kv * hd * sum(lens) + 4 * 4097,
            "flops": 4 * pairs * c["heads"] * hd}


# ------------------------------------------------------------------ inputs

def _exp_table():
    return [int(math.floor(math.exp(-i / 256.0) * 2.0**30 + 0.5)) for i in range(4097)]


def _normal(shape, g, sigma):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).round().to(torch.int64)


def _pool(c, pages, g):
    """Words of unit spread, as normalised keys and values are."""
    shape = (pages, c["layers"], c["kv_heads"], c["page"], c["head"])
    return (torch.randn(shape, generator=g, device="cuda") * 65536.0).round().to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "beam":
        rows = c["groups"] * c["beams"]
        s["logits"] = _normal((rows, c["vocab"]), g, 3 * 65536.0)
        # sums of log-probabilities some steps into a search; a few beams have ended, one is dead
        scores = -torch.randint(0, 40 << 16, (rows,), generator=g, device="cuda")
        u = torch.rand(rows, generator=g, device="cuda")
        s["done"] = (u < 0.1).to(torch.uint8)
        s["scores"] = torch.where(u > 0.95, torch.full_like(scores, MIN), scores)
        s["exp"] = torch.tensor(_exp_table(), device="cuda")
        if own:
            import fixed_point_int8_gb300 as ck
            s["exp32"] = s["exp"].to(torch.int32)
            s["plan"] = ck.BeamPlan(c["groups"], c["beams"], c["vocab"])
        return s
    page = c["page"]
    if c["op"] in ("fork", "compact"):
        lens, pages, shared = _row_pages(c)
        rows, stride = len(lens), max(pages) + 2
        held, total = _pages_held(c)
        ids = torch.randperm(total, generator=g, device="cuda")[:held].tolist()
        table, group = [], []
        for r in range(rows):
            if r % c["beams"] == 0:
                group, ids = ids[:shared[r]], ids[shared[r]:]
            mine = pages[r] - shared[r]
            table.append(group + ids[:mine] + [-1] * (stride - pages[r]))
            ids = ids[mine:]
        s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = _pool(c, total, g), _pool(c, total, g)
        if c["op"] == "fork":
            # what a step of a search asks for: parents of the own group, better beams more often
            u = torch.rand(rows, generator=g, device="cuda")
            first = torch.arange(rows, device="cuda") // c["beams"] * c["beams"]
            s["parent"] = (first + (u * u * c["beams"]).long().clamp(max=c["beams"] - 1)).to(torch.int32)
            s["grow"] = torch.ones(rows, dtype=torch.int32, device="cuda")
        if own:
            import fixed_point_int8_gb300 as ck
            s["cache"] = ck.PagedCache(s["k"], s["v"])
            s["plan"] = ck.PagePlan(s["cache"], rows, stride)
        return s
    lens, news = _lens(c), _news(c)
    stride = -(-max(lens) // page) + 1
    pages = sum(-(-n // page) for n in lens)
    ids = torch.randperm(pages + 1, generator=g, device="cuda").tolist()
    table = []
    for n in lens:
        m = -(-n // page)
        table.append(ids[:m] + [-1] * (stride - m))
        ids = ids[m:]
    rows = sum(news)
    s["rows"], s["new"], s["len"] = rows, max(news), max(lens)
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32, device="cuda")
    s["status"] = torch.full((len(lens),), -1, dtype=torch.int64, device="cuda")
    s["k"], s["v"] = _pool(c, pages + 1, g), _pool(c, pages + 1, g)
    q_dim, kv_dim = c["heads"] * c["head"], c["kv_heads"] * c["head"]
    s["out"] = torch.zeros(rows, q_dim, dtype=torch.int64, device="cuda")
    if c["op"] == "attend":
        s["q"] = _normal((rows, q_dim), g, 65536.0)
        s["exp"] = torch.tensor(_exp_table(), device="cuda")
        s["inv"] = int(math.floor(2.0**24 / math.sqrt(c["head"]) + 0.5))
    else:
        # the stacked matrix rows of a layer: queries, keys and values of a row side by side
        s["qkv"] = _normal((rows, q_dim + 2 * kv_dim), g, 65536.0)
        angle = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
            -2.0 * torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) / c["rot"])
        s["rope"] = (torch.stack((angle.cos(), angle.sin()), -1) * 2.0**24).round().to(torch.int32)
    if own:
        import fixed_point_int8_gb300 as ck
        s["cache"] = ck.PagedCache(s["k"], s["v"])
        s["batch"] = ck.PagedBatch(s["table"], s["lens"], s["starts"], s["status"], rows, s["new"], s["len"])
        if c["op"] == "attend":
            s["exp32"] = s["exp"].to(torch.int32)
            s["work"] = ck.paged_attention_work(s["cache"], s["batch"], c["heads"])
    return s


# ------------------------------------------------------------------ plain forms

def _rows_of(s):
    """Of each sequence (padded to the most new tokens): which slots are rows, the rows' numbers
    (one past the last where there is none) and their positions."""
    starts, lens = s["starts"].long(), s["lens"].long()
    j = torch.arange(s["new"], device=lens.device)
    n = starts[1:] - starts[:-1]
    pos = (lens - n)[:, None] + j
    valid = (j < n[:, None]) & (pos >= 0)
    return valid, torch.where(valid, starts[:-1, None] + j, s["rows"]), pos


def _attend(s):
    c, dev = s["case"], s["q"].device
    kv, hd, page = c["kv_heads"], c["head"], c["page"]
    group = c["heads"] // kv
    valid, row, pos = _rows_of(s)
    t = torch.arange(s["len"], device=dev)
    at = s["table"].long()[:, t // page].clamp(min=0)
    k = s["k"][:, 0][at, :, (t % page)[None, :]].long().transpose(1, 2)     # [seq][kv][t][hd]
    v = s["v"][:, 0][at, :, (t % page)[None, :]].long().transpose(1, 2)
    q = s["q"][row.clamp(max=s["rows"] - 1)].view(*row.shape, kv, group, 1, hd)
    dot = (q * k[:, None, :, None]).sum(-1)                                  # [seq][row][kv][group][t]
    score = ((dot >> 16) * s["inv"]) >> 24
    mask = ((t <= pos[..., None]) & valid[..., None])[:, :, None, None]
    m = torch.where(mask, score, MIN).amax(-1, keepdim=True)
    low = torch.where(m > MIN + 2**40, m - 2**40, MIN)
    index = ((m - torch.maximum(score, low)) >> 8).clamp(0, 4096)
    e = s["exp"][index] * mask
    z = e.sum(-1, keepdim=True)
    p = (e << 24) // z.clamp(min=2**30)
    o = (p[..., None] * v[:, None, :, None]).sum(-2) >> 24                   # [seq][row][kv][group][hd]
    out = torch.zeros(s["rows"] + 1, c["heads"] * hd, dtype=torch.int64, device=dev)
    out[row.reshape(-1)] = o.reshape(-1, c["heads"] * hd)
    return {"out": out[:-1], "status": s["status"]}


def _rotate(x, cs, rot, half):
    """x [..., head]; cs [..., rot / 2, 2]."""
    c, sn = cs[..., 0], cs[..., 1]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    a2, b2 = (a * c - b * sn) >> 24, (a * sn + b * c) >> 24
    turned = torch.cat((a2, b2), -1) if half else torch.stack((a2, b2), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _store(s):
    c, dev = s["case"], s["qkv"].device
    kv, hd, page, rot = c["kv_heads"], c["head"], c["page"], c["rot"]
    starts, lens = s["starts"].long(), s["lens"].long()
    row = torch.arange(s["rows"], device=dev)
    seq = (row[:, None] >= starts[None, 1:]).sum(-1)
    pos = lens[seq] - starts[seq + 1] + row
    cs = s["rope"].long()[pos][:, None]
    q_dim, kv_dim = c["heads"] * hd, kv * hd
    q, k, v = s["qkv"].split((q_dim, kv_dim, kv_dim), -1)
    q = _rotate(q.view(-1, c["heads"], hd), cs, rot, c["half"]).flatten(1)
    k = k.reshape(-1, kv, hd)
    turned = _rotate(k.to(torch.int32).long(), cs, rot, c["half"])
    v = v.reshape(-1, kv, hd)
    # the smallest (position, phase, element) whose word does not fit 32 bits, per sequence
    element = torch.arange(kv_dim, device=dev).view(kv, hd)

    def first(x, phase):
        key = (pos[:, None, None] << 44) | (phase << 24) | element
        return torch.where(x != x.to(torch.int32), key, 2**63 - 1).amin((1, 2))

    key = torch.minimum(torch.minimum(first(k, 6), first(v, 7)), first(turned, 8))
    worst = torch.full_like(lens, 2**63 - 1).scatter_reduce(0, seq, key, "amin")
    status = torch.where(worst == 2**63 - 1, s["status"], worst)
    at = s["table"].long()[seq, pos // page]
    s["k"][:, 0].transpose(1, 2)[at, pos % page] = turned.to(torch.int32)
    s["v"][:, 0].transpose(1, 2)[at, pos % page] = v.to(torch.int32)
    return {"q": q, "k": s["k"], "v": s["v"], "status": status}


def _fork(s):
    c, dev = s["case"], s["table"].device
    page, pages = c["page"], s["k"].shape[0]
    table, parent = s["table"].long(), s["parent"].long()
    rows, stride = table.shape
    col = torch.arange(stride, device=dev)
    row = torch.arange(rows, device=dev)
    old = s["lens"].long()[parent]
    length = old + s["grow"].long()
    full, part = old // page, old % page
    kept = torch.where(col < full[:, None], table[parent], -1)
    last = torch.where(part > 0, table[parent, full.clamp(max=stride - 1)], pages)   # `pages`: none
    # a part-filled page stays with its first holder, unless another row has it whole
    owner = torch.full((pages + 1,), rows, device=dev).scatter_reduce(0, last, row, "amin")
    used = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    used[torch.where(kept >= 0, kept, pages)] = True
    stays = (part > 0) & (owner[last] == row) & ~used[last]
    taken = used.clone()
    taken[torch.where(stays, last, pages)] = True
    # the free pages go out in ascending order, row after row
    have = full + stays
    need = (length + page - 1) // page - have
    before = need.cumsum(0) - need
    taken[pages] = True
    free = torch.sort(taken.to(torch.int8), stable=True)[1]
    served = before + need <= (~taken).sum()
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    nth = (before[:, None] + col - have[:, None]).clamp(0, pages)
    new = torch.where(stays[:, None] & (col == full[:, None]), last[:, None], kept)
    new = torch.where(fresh, free[nth], new)
    new = torch.where(served[:, None], new, -1)
    # copies: the filled positions of the part-filled pages that stay with another row
    moved = (part > 0) & ~stays & served
    slot = torch.arange(page, device=dev)
    mask = (moved[:, None] & (slot < part[:, None]))[:, None, None, :, None]
    # rows that copy nothing write a taken page's own words: no copy's target is a taken page
    idle = taken[:-1].to(torch.int8).argmax()
    src = torch.where(moved, last, idle)
    target = torch.where(moved, new[row, full.clamp(max=stride - 1)], idle)
    s["k"][target] = torch.where(mask, s["k"][src], s["k"][target])
    s["v"][target] = torch.where(mask, s["v"][src], s["v"][target])
    return {"table": new.to(torch.int32), "lens": torch.where(served, length, 0).to(torch.int32),
            "status": torch.where(served, 0, 4).to(torch.int32), "k": s["k"], "v": s["v"]}


def _compact(s):
    c, dev = s["case"], s["table"].device
    pages, table = s["k"].shape[0], s["table"].long()
    rows, stride = table.shape
    col = torch.arange(stride, device=dev)
    inside = col < ((s["lens"].long() + c["page"] - 1) // c["page"])[:, None]
    used = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    used[torch.where(inside, table, pages)] = True
    used = used[:-1]
    count = used.sum()
    ident = torch.arange(pages, device=dev)
    low = ident < count
    movers, holes = used & ~low, ~used & low
    rank = movers.cumsum(0) - 1
    hole = torch.sort((~holes).to(torch.int8), stable=True)[1]
    to = torch.where(movers, hole[rank.clamp(min=0)], ident)
    source = torch.arange(pages + 1, device=dev)
    source[torch.where(used, to, pages)] = ident
    s["k"][:] = s["k"][source[:-1]]
    s["v"][:] = s["v"][source[:-1]]
    new = torch.where(inside, to[table.clamp(min=0)], -1)
    return {"table": new.to(torch.int32), "used": count.to(torch.int32), "status": torch.zeros_like(s["lens"]),
            "k": s["k"], "v": s["v"]}


def _ln(z):
    """ln(z / 2^30) for z >= 2^30, with 16 fraction bits: z = 2^n y, ln y = 2 atanh((y - 1) / (y + 1))."""
    z = z.clamp(min=2**30)
    power = torch.tensor([2**(31 + i) for i in range(24)], device=z.device)
    n = (z[:, None] >= power).sum(-1)
    y = z >> n
    t = ((y - 2**30) << 30) // (y + 2**30)
    t2 = (t * t) >> 30
    # the series' coefficients 2^30 / (2 i + 1), from i = 7 down
    p = 82595525 + ((71582788 * t2) >> 30)
    p = 97612893 + ((p * t2) >> 30)
    p = 119304647 + ((p * t2) >> 30)
    p = 153391689 + ((p * t2) >> 30)
    p = 214748365 + ((p * t2) >> 30)
    p = 357913941 + ((p * t2) >> 30)
    p = 1073741824 + ((p * t2) >> 30)
    return (n * LN2 + 2 * ((t * p) >> 30) + 2**13) >> 14


def _beam(s):
    c, dev = s["case"], s["logits"].device
    groups, beams, vocab = c["groups"], c["beams"], c["vocab"]
    logits, old, done = s["logits"], s["scores"], s["done"].bool()
    alive = (old > DEAD) & (old < -DEAD)
    m = logits.amax(-1, keepdim=True)
    low = torch.where(m > MIN + 2**62, m - 2**62, MIN)
    d = m - torch.maximum(logits, low)
    z = s["exp"][(d >> 8).clamp(max=4096)].sum(-1)
    score = (old - _ln(z))[:, None] - d
    score = torch.where((alive & ~done)[:, None], score, MIN)
    # an ended beam is one candidate, behind its own vocabulary; token 2 is what it carries on with
    ended = torch.where(alive & done, old, MIN)[:, None]
    score = torch.cat((score, ended), -1).view(groups, beams * (vocab + 1))
    best, at = torch.sort(score, dim=-1, descending=True, stable=True)
    best, at = best[:, :beams].flatten(), at[:, :beams].flatten()
    first = torch.arange(groups * beams, device=dev) // beams * beams
    some = best != MIN
    token = at % (vocab + 1)
    carried = some & (token == vocab)
    parent = torch.where(some, first + at // (vocab + 1), NO_ROW)
    token = torch.where(some & ~carried, token, min(2, vocab - 1))
    stops = carried | (some & ((token == 1) | (token == 2)))
    return {"scores": best, "parent": parent.to(torch.int32), "token": token.to(torch.int32),
            "done": stops.to(torch.uint8)}


def exact(case, seed):
    """The same from the definitions on the host: numpy on 64-bit words, and Python's integers."""
    import numpy as np
    c = case
    s = prepare(case, seed)
    h = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor)}

    def product(a, b):
        """a @ b modulo 2^64: 15-bit pieces, whose double-precision products are exact."""
        total = np.zeros((a.shape[0], b.shape[1]), dtype=np.uint64)
        for i in range(0, 64, 15):
            x = (a >> i) if i == 60 else ((a >> i) & 0x7FFF)
            for j in range(0, 64 - i, 15):
                y = (b >> j) if j == 60 else ((b >> j) & 0x7FFF)
                if x.any() and y.any():
                    part = x.astype(np.float64) @ y.astype(np.float64)
                    total += part.astype(np.int64).astype(np.uint64) << np.uint64(i + j)
        return total.view(np.int64)

    if c["op"] == "attend":
        if 16 * work(c)["flops"] > 3e11:
            return None
        hd, group, page = c["head"], c["heads"] // c["kv_heads"], c["page"]
        table = np.array(_exp_table(), dtype=np.int64)
        out = np.zeros((s["rows"], c["heads"] * hd), dtype=np.int64)
        for i, (n, length) in enumerate(zip(_news(c), _lens(c))):
            r0 = int(h["starts"][i])
            where = [(int(h["table"][i, t // page]), t % page) for t in range(length)]
            pg, sl = np.array(where, dtype=np.int64).reshape(-1, 2).T
            for kvh in range(c["kv_heads"]):
                kk = h["k"][pg, 0, kvh, sl].astype(np.int64)
                vv = h["v"][pg, 0, kvh, sl].astype(np.int64)
                for head in range(kvh * group, (kvh + 1) * group):
                    q = h["q"][r0:r0 + n, head * hd:(head + 1) * hd]
                    score = ((product(q, kk.T.copy()) >> 16) * s["inv"]) >> 24
                    seen = np.arange(length)[None, :] <= (length - n + np.arange(n))[:, None]
                    m = np.where(seen, score, MIN).max(-1, keepdims=True)
                    e = np.where(seen, table[np.minimum((m - np.minimum(score, m)) >> 8, 4096)], 0)
                    p = (e << 24) // e.sum(-1, keepdims=True)
                    out[r0:r0 + n, head * hd:(head + 1) * hd] = product(p, vv) >> 24
        return {"out": out, "status": h["status"]}
    if c["op"] == "store":
        hd, kv, page, rot = c["head"], c["kv_heads"], c["page"], c["rot"]
        heads, qkv = c["heads"] + kv, h["qkv"]
        turned = qkv[:, :heads * hd].copy()
        k, v = h["k"].copy(), h["v"].copy()
        pairs = [(j, j + rot // 2) if c["half"] else (2 * j, 2 * j + 1) for j in range(rot // 2)]
        for i, (n, length) in enumerate(zip(_news(c), _lens(c))):
            for j in range(n):
                r, pos = int(h["starts"][i]) + j, length - n + j
                for x in range(rot // 2):
                    co, si = (int(w) for w in h["rope"][pos, x])
                    a, b = qkv[r, pairs[x][0]:heads * hd:hd], qkv[r, pairs[x][1]:heads * hd:hd]
                    turned[r, pairs[x][0]::hd] = (a * co - b * si) >> 24
                    turned[r, pairs[x][1]::hd] = (a * si + b * co) >> 24
                pg, sl = int(h["table"][i, pos // page]), pos % page
                k[pg, 0, :, sl] = turned[r, c["heads"] * hd:].reshape(kv, hd)
                v[pg, 0, :, sl] = qkv[r, heads * hd:].reshape(kv, hd)
        return {"q": turned[:, :c["heads"] * hd], "k": k, "v": v, "status": h["status"]}
    if c["op"] == "fork":
        page, rows, stride = c["page"], *h["table"].shape
        old = [int(h["lens"][p]) for p in h["parent"]]
        kept = [[int(w) for w in h["table"][p][:n // page]] for p, n in zip(h["parent"], old)]
        used = {w for row in kept for w in row}
        holder = {}
        for r in range(rows):
            if old[r] % page:
                w = int(h["table"][h["parent"][r], old[r] // page])
                if w not in used and holder.setdefault(w, r) == r:
                    kept[r].append(w)
        used |= set(holder)
        free = [w for w in range(h["k"].shape[0]) if w not in used]
        asked, status, lens = 0, [], []
        for r in range(rows):
            length = old[r] + int(h["grow"][r])
            need = -(-length // page) - len(kept[r])
            ok = asked + need <= len(free)
            kept[r] = kept[r] + free[asked:asked + need] if ok else []
            asked += need
            status.append(0 if ok else 4)
            lens.append(length if ok else 0)
        table = np.array([row + [-1] * (stride - len(row)) for row in kept], dtype=np.int32)
        return {"table": table, "lens": np.array(lens, dtype=np.int32), "status": np.array(status, dtype=np.int32),
                "k": None, "v": None}
    if c["op"] == "compact":
        page, rows, stride = c["page"], *h["table"].shape
        mine = [[int(w) for w in h["table"][r][:-(-int(h["lens"][r]) // page)]] for r in range(rows)]
        used = sorted({w for row in mine for w in row})
        holes = [w for w in range(len(used)) if w not in set(used)]
        to = {w: w for w in used if w < len(used)}
        to.update(zip((w for w in used if w >= len(used)), holes))
        table = np.array([[to[w] for w in row] + [-1] * (stride - len(row)) for row in mine], dtype=np.int32)
        return {"table": table, "used": np.int32(len(used)), "status": np.zeros(rows, dtype=np.int32),
                "k": None, "v": None}
    groups, beams, vocab = c["groups"], c["beams"], c["vocab"]
    table = np.array(_exp_table(), dtype=np.int64)
    scores, parent, token, done = [], [], [], []
    for g in range(groups):
        found = []
        for r in range(g * beams, (g + 1) * beams):
            old = int(h["scores"][r])
            if not DEAD < old < -DEAD:
                continue
            if h["done"][r]:
                found.append((-old, r, vocab))
                continue
            d = h["logits"][r].max() - h["logits"][r]
            z = int(table[np.minimum(d >> 8, 4096)].sum())
            n = z.bit_length() - 31
            y = z >> n
            t = ((y - 2**30) << 30) // (y + 2**30)
            t2, p = (t * t) >> 30, 0
            for i in range(7, -1, -1):
                p = (2**31 // (2 * i + 1) + 1) // 2 + ((p * t2) >> 30)
            ln = (n * LN2 + 2 * ((t * p) >> 30) + 2**13) >> 14
            order = np.argsort(d, kind="stable")[:beams]
            found += [(int(d[w]) + ln - old, r, int(w)) for w in order]
        found = sorted(found)[:beams]
        for cost, r, w in found:
            scores.append(-cost)
            parent.append(r)
            token.append(min(2, vocab - 1) if w == vocab else w)
            done.append(int(w == vocab or w in (1, 2)))
        for _ in range(beams - len(found)):
            scores.append(MIN)
            parent.append(NO_ROW)
            token.append(min(2, vocab - 1))
            done.append(0)
    return {"scores": np.array(scores, dtype=np.int64), "parent": np.array(parent, dtype=np.int32),
            "token": np.array(token, dtype=np.int32), "done": np.array(done, dtype=np.uint8)}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"attend": _attend, "store": _store, "fork": _fork, "compact": _compact, "beam": _beam}[op](s)
    import fixed_point_int8_gb300 as ck
    c = s["case"]
    if op == "attend":
        rc, out = ck.paged_attention(s["cache"], 0, s["batch"], s["q"], s["exp32"], s["inv"], out=s["out"],
                                     work=s["work"])
        result = {"out": out, "status": s["status"]}
    elif op == "store":
        q_dim, kv_dim = c["heads"] * c["head"], c["kv_heads"] * c["head"]
        q, k, v = s["qkv"].split((q_dim, kv_dim, kv_dim), -1)
        rc, q = ck.paged_store(s["cache"], 0, s["batch"], q, k, v, s["rope"], half=c["half"], out=s["out"])
        result = {"q": q, "k": s["k"], "v": s["v"], "status": s["status"]}
    elif op == "fork":
        rc, got = s["plan"].fork(s["parent"], s["lens"], s["table"], s["grow"])
        result = {"table": got.table, "lens": got.lens, "status": got.status, "k": s["k"], "v": s["v"]}
    elif op == "compact":
        rc, got = s["plan"].compact(s["lens"], s["table"])
        result = {"table": got.table, "used": got.used, "status": got.status, "k": s["k"], "v": s["v"]}
    else:
        rc, got = s["plan"].select(s["logits"], s["scores"], s["done"], s["exp32"], stop_tokens=True,
                                   done_token=min(2, c["vocab"] - 1))
        result = {"scores": got.scores, "parent": got.parent, "token": got.token, "done": got.done}
    if rc:
        raise RuntimeError("%s: error %d" % (op, rc))
    return result
