"""The operators of long streams served together, as they are measured: attention over a window and
a few first positions that stay visible, the page tables' step between passes, and sampling.  Their
cases, inputs and plain forms in elementary torch operations on 64-bit integers.

Formats are the library's: queries, logits and scores are int64 with 16 fraction bits, cached words
int32 with 16, temperatures u32 with 16, the exponential table 4,097 entries with 30, probabilities
and their thresholds u32 with 24.  A pool is int32 [pages][layers][kv heads][page][head]; a table row
lists a sequence's pages in order, -1 where there is none."""
import math

import torch

own = False

MIN = -2**63           # a masked logit
FAR = 2**62
ONE = 2**24            # a probability of one
LONGEST = 2**20 - 1    # positions of a sequence


def listed():
    return [
        # one stream of the 1B shape late in its 8K context, a single new token: the last 2,048
        # positions and the first four
        {"name": "window_1b_8191", "op": "window", "seqs": 1, "new": 1, "len_min": 8191, "len": 8191, "sinks": 4,
         "window": 2048, "heads": 32, "kv_heads": 32, "head": 64, "page": 64},
        # 64 streams of the 1B shape, each at a position of its own, one new token a stream
        {"name": "window_1b_64streams", "op": "window", "seqs": 64, "new": 1, "len_min": 901, "len": 8191, "sinks": 4,
         "window": 1024, "heads": 32, "kv_heads": 32, "head": 64, "page": 16},
        # chunks of two prompts of the 7B shape, ragged in new tokens and in length
        {"name": "window_7b_chunk", "op": "window", "seqs": 2, "new": 201, "len_min": 777, "len": 2047, "sinks": 4,
         "window": 509, "heads": 32, "kv_heads": 32, "head": 128, "page": 32},
        # the last chunk of a long prompt of the 1B shape
        {"name": "window_1b_chunk_7936", "op": "window", "seqs": 1, "new": 256, "len_min": 7936, "len": 7936,
         "sinks": 4, "window": 2048, "heads": 32, "kv_heads": 32, "head": 64, "page": 64},
        # a small grouped-head model's four streams between two passes
        {"name": "advance_gqa_4", "op": "advance", "seqs": 4, "len_min": 30, "len": 97, "chunk": 1, "sinks": 4,
         "window": 40, "page": 16, "context": 512, "spare": 9, "held": False},
        # 64 streams of the 1B shape in its 8K context: every one has a new token, pages behind the
        # windows come back
        {"name": "advance_1b_64", "op": "advance", "seqs": 64, "len_min": 901, "len": 8190, "chunk": 1, "sinks": 4,
         "window": 1024, "page": 16, "context": 8192, "spare": 64, "held": True},
        # a full server: 2,048 sequences of the 1B shape's context without a window, one in eight with
        # a chunk of its prompt
        {"name": "advance_2048", "op": "advance", "seqs": 2048, "len_min": 65, "len": 1901, "chunk": 33, "sinks": 0,
         "window": 0, "page": 16, "context": 2048, "spare": 4001, "held": True},
        # one run's next token over the vocabulary, with every filter
        {"name": "sample_1", "op": "sample", "rows": 1, "vocab": 32000, "k": True, "p": True, "m": True},
        # the small model's eight runs, temperature and nucleus only
        {"name": "sample_gqa_8", "op": "sample", "rows": 8, "vocab": 512, "k": False, "p": True, "m": False},
        # 64 runs of the 1B shape, each with settings of its own
        {"name": "sample_64", "op": "sample", "rows": 64, "vocab": 32000, "k": True, "p": True, "m": True},
        # 512 runs by temperature alone, and 512 with a nucleus and the least probability
        {"name": "sample_512_plain", "op": "sample", "rows": 512, "vocab": 32000, "k": False, "p": False, "m": False},
        {"name": "sample_512", "op": "sample", "rows": 512, "vocab": 32000, "k": False, "p": True, "m": True},
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["window", "window", "advance", "sample"])
    if op == "sample":
        return {"op": op, "rows": log(1, 512), "vocab": log(7, 32000), "k": rng.random() < 0.6,
                "p": rng.random() < 0.6, "m": rng.random() < 0.6}
    c = {"op": op, "page": rng.choice([8, 16, 32, 64]), "sinks": rng.choice([0, 1, 4, rng.randint(0, 70)])}
    if op == "advance":
        c["seqs"] = log(1, 2048)
        c["len"] = log(9, 8190 if c["seqs"] <= 64 else 1901)
        c["len_min"] = rng.randint(0, c["len"])
        many = c["seqs"] > 64
        c["page"] = max(c["page"], 16) if many else c["page"]
        c["chunk"] = rng.choice([1, log(1, 33 if many else 250)])
        c["window"] = rng.choice([0, log(1, c["len"])])     # 0: everything stays
        c["context"] = c["len"] + rng.choice([c["chunk"], rng.randint(0, 147 if many else 600)])
        # some pools are too small for what the sequences ask for
        c["spare"] = rng.choice([log(1, 2 * c["seqs"]), c["seqs"] * (2 + c["chunk"] // c["page"])])
        c["held"] = rng.random() < 0.5
        return c
    c["head"] = rng.choice([4, 8, 16, 32, 64, 128])
    c["kv_heads"] = rng.choice([1, 2, 4, 8, 32 if c["head"] <= 64 else 8])
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 4] if c["kv_heads"] <= 8 else [1])
    if rng.random() < 0.5:
        c.update(seqs=log(1, 64), new=1, window=log(1, 950))
        c["len"] = log(1, 8191)
    else:
        c.update(seqs=rng.randint(1, 2), new=log(2, 201), window=log(1, 600))
        c["len"] = c["new"] + rng.randint(0, 6000)
    c["len_min"] = rng.randint((c["len"] + 1) // 2, c["len"])
    return c


# ------------------------------------------------------------------ sizes

def _lens(c):
    """Positions of each sequence, from the least to the most (of a window's case with the new ones)."""
    n = c["seqs"]
    return [c["len"] - (c["len"] - c["len_min"]) * i // max(1, n - 1) for i in range(n)]


def _news(c):
    """New tokens of each sequence: the first has c["new"], the others less."""
    return [max(1, min(n, c["new"] - (c["new"] * i) // (2 * c["seqs"]))) for i, n in enumerate(_lens(c))]


def _asks(c):
    """New tokens each sequence asks for: one, and a chunk for the first and every eighth after."""
    return [1 if i % 8 else c["chunk"] for i in range(c["seqs"])]


def _kept_pages(c):
    """Of each sequence the numbers, from its start, of the pages that the step keeps."""
    page, out = c["page"], []
    for n in _lens(c):
        have = -(-n // page)
        if not c["window"]:
            out.append(list(range(have)))
        else:
            out.append([i for i in range(have) if i * page < c["sinks"] or (i + 1) * page + c["window"] > n + 1])
    return out


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        return {"bytes": 8 * n + 4 * 4097 + c["rows"] * (24 + 4 * (c["k"] + c["p"] + c["m"])), "flops": 4 * n}
    if c["op"] == "advance":
        kept, stride = sum(len(k) for k in _kept_pages(c)), -(-c["context"] // c["page"])
        pages = kept + c["spare"]
        return {"bytes": 4 * kept + 4 * c["seqs"] * stride + (pages if c["held"] else 0) + 20 * c["seqs"]
                + 12 * sum(_asks(c)), "flops": pages}
    hd, kv, rows, seen, pairs = c["head"], c["kv_heads"], sum(_news(c)), 0, 0
    for n, length in zip(_news(c), _lens(c)):
        low = max(0, length - n - c["window"] + 1)
        seen += length - low + min(c["sinks"], low)
        for pos in range(length - n, length):
            behind = max(0, pos + 1 - c["window"])
            pairs += pos + 1 - behind + min(c["sinks"], behind)
    return {"bytes": 16 * rows * c["heads"] * hd + 8 * kv * hd * seen + 4 * 4097, "flops": 4 * pairs * c["heads"] * hd}


# ------------------------------------------------------------------ inputs

def _exp_table():
    return [int(math.floor(math.exp(-i / 256.0) * 2.0**30 + 0.5)) for i in range(4097)]


def _normal(shape, g, sigma):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).round().to(torch.int64)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "sample":
        rows, vocab = c["rows"], c["vocab"]
        s["logits"] = _normal((rows, vocab), g, 3 * 65536.0)
        # a run in sixteen follows a grammar that allows about a third of the vocabulary
        u = torch.rand(rows, generator=g, device="cuda")
        bound = torch.rand((rows, vocab), generator=g, device="cuda") > 0.35
        s["logits"].masked_fill_(bound & (u < 1 / 16)[:, None], MIN)
        # temperatures from 0.3 to 1.5, a run in ten takes the largest logit; top-k to 200, or all;
        # nuclei from 0.5 to 0.99, or all; least probabilities to 0.1 of the largest, or none
        t = (0.3 + 1.2 * torch.rand(rows, generator=g, device="cuda")) * 65536
        off = torch.rand((4, rows), generator=g, device="cuda")
        part = torch.rand((3, rows), generator=g, device="cuda")
        s["temperature"] = torch.where(off[0] < 0.1, torch.zeros_like(t), t).to(torch.int32)
        top_k = torch.where(off[1] < 0.25, torch.zeros_like(t), 1 + part[0] * 199).to(torch.int32)
        top_p = torch.where(off[2] < 0.25, torch.full_like(t, ONE), (0.5 + 0.49 * part[1]) * ONE).to(torch.int32)
        min_p = torch.where(off[3] < 0.25, torch.zeros_like(t), (0.01 + 0.09 * part[2]) * ONE).to(torch.int32)
        s["top_k"], s["top_p"], s["min_p"] = top_k if c["k"] else None, top_p if c["p"] else None, min_p if c["m"] else None
        s["random"] = torch.randint(-2**63, 2**63 - 1, (rows,), generator=g, device="cuda")
        s["exp"] = _i32(_exp_table())
        return s
    page, lens = c["page"], _lens(c)
    if c["op"] == "advance":
        kept, stride = _kept_pages(c), -(-c["context"] // page)
        # the pages of the step before: one more behind each window's
        before = []
        for n, mine in zip(lens, kept):
            gone = [i for i in range(-(-n // page)) if i not in set(mine)][-1:]
            before.append(sorted(mine + gone))
        total = sum(map(len, kept)) + c["spare"] + (c["spare"] // 8 if c["held"] else 0)
        total = max(total, sum(map(len, before)))
        ids = torch.randperm(total, generator=g, device="cuda").tolist()
        table, at = [[-1] * stride for _ in lens], 0
        for row, mine in zip(table, before):
            for i in mine:
                row[i] = ids[at]
                at += 1
        s["table"], s["lens"], s["new"] = _i32(table), _i32(lens), _i32(_asks(c))
        s["rows"] = sum(_asks(c))
        s["held"] = None
        if c["held"]:  # prompts that are kept for later
            s["held"] = torch.zeros(total, dtype=torch.uint8, device="cuda")
            s["held"][_i32(ids[at:at + c["spare"] // 8]).long()] = 1
        s["pages"] = total
        if own:
            import fixed_point_int8_gb300 as ck
            s["cache"] = ck.PagedCache.empty(total, 1, 1, page, 4)
            s["plan"] = ck.PagePlan(s["cache"], c["seqs"], stride)
        return s
    news, stride, at, table = _news(c), -(-max(lens) // page) + 1, 0, []
    seen = []
    for n, length in zip(news, lens):
        low = max(0, length - n - c["window"] + 1)
        seen.append([i for i in range(-(-length // page)) if i * page < c["sinks"] or (i + 1) * page > low])
    pages = sum(map(len, seen)) + 1
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    for mine in seen:  # pages that no row sees have been given back
        row = [-1] * stride
        for i in mine:
            row[i] = ids[at]
            at += 1
        table.append(row)
    rows = sum(news)
    s["rows"], s["new"], s["len"] = rows, max(news), max(lens)
    s["table"], s["lens"] = _i32(table), _i32(lens)
    s["starts"] = _i32([sum(news[:i]) for i in range(len(news) + 1)])
    s["status"] = torch.full((len(lens),), -1, dtype=torch.int64, device="cuda")
    shape = (pages, 1, c["kv_heads"], page, c["head"])
    s["k"], s["v"] = ((torch.randn(shape, generator=g, device="cuda") * 65536.0).round().to(torch.int32) for _ in "kv")
    s["q"] = _normal((rows, c["heads"] * c["head"]), g, 65536.0)
    s["out"] = torch.zeros(rows, c["heads"] * c["head"], dtype=torch.int64, device="cuda")
    s["exp"] = _i32(_exp_table())
    s["inv"] = int(math.floor(2.0**24 / math.sqrt(c["head"]) + 0.5))
    if own:
        import fixed_point_int8_gb300 as ck
        s["cache"] = ck.PagedCache(s["k"], s["v"])
        s["batch"] = ck.PagedBatch(s["table"], s["lens"], s["starts"], s["status"], rows, s["new"], s["len"])
        s["view"] = ck.Window(c["sinks"], c["window"])
        s["work"] = ck.paged_attention_work(s["cache"], s["batch"], c["heads"], window=s["view"])
    return s


# ------------------------------------------------------------------ plain forms

def _window(s):
    c, dev = s["case"], s["q"].device
    kv, hd, page, sinks, window = c["kv_heads"], c["head"], c["page"], c["sinks"], c["window"]
    group = c["heads"] // kv
    starts, lens = s["starts"].long(), s["lens"].long()
    # of each sequence (padded to the most new tokens): which slots are rows, their numbers (one past
    # the last where there is none) and their positions
    j = torch.arange(s["new"], device=dev)
    n = starts[1:] - starts[:-1]
    pos = (lens - n)[:, None] + j
    valid = (j < n[:, None]) & (pos >= 0)
    row = torch.where(valid, starts[:-1, None] + j, s["rows"])
    # the positions that any row of the sequence sees: the first ones, then those of the windows
    low = (lens - n - window + 1).clamp(min=sinks)
    t = torch.cat((torch.arange(sinks, device=dev).expand(len(lens), -1),
                   low[:, None] + torch.arange(window + s["new"] - 1, device=dev)), 1)
    at = s["table"].long().gather(1, (t // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k = s["k"][:, 0][at, :, t % page].long().transpose(1, 2)                 # [seq][kv][t][hd]
    v = s["v"][:, 0][at, :, t % page].long().transpose(1, 2)
    q = s["q"][row.clamp(max=s["rows"] - 1)].view(*row.shape, kv, group, 1, hd)
    dot = (q * k[:, None, :, None]).sum(-1)                                  # [seq][row][kv][group][t]
    score = ((dot >> 16) * s["inv"]) >> 24
    u, p = t[:, None], pos[..., None]
    mask = ((u <= p) & ((u < sinks) | (u > p - window)) & valid[..., None])[:, :, None, None]
    m = torch.where(mask, score, MIN).amax(-1, keepdim=True)
    low = torch.where(m > MIN + 2**40, m - 2**40, MIN)
    index = ((m - torch.maximum(score, low)) >> 8).clamp(0, 4096)
    e = s["exp"].long()[index] * mask
    z = e.sum(-1, keepdim=True)
    p = (e << 24) // z.clamp(min=2**30)
    o = (p[..., None] * v[:, None, :, None]).sum(-2) >> 24                   # [seq][row][kv][group][hd]
    out = torch.zeros(s["rows"] + 1, c["heads"] * hd, dtype=torch.int64, device=dev)
    out[row.reshape(-1)] = o.reshape(-1, c["heads"] * hd)
    return {"out": out[:-1], "status": s["status"]}


def _advance(s):
    c, dev = s["case"], s["table"].device
    page, pages, sinks, window = c["page"], s["pages"], c["sinks"], c["window"]
    table, lens, new = s["table"].long(), s["lens"].long(), s["new"].long()
    seqs, stride = table.shape
    i = torch.arange(stride, device=dev)
    have = (lens + page - 1) // page
    keep = i < have[:, None]
    if window:
        keep &= (i * page < sinks) | ((i + 1) * page + window > lens[:, None] + 1)
    # 3: a kept page outside the pool, or a length that the table does not hold; 7: too long
    lost = (lens > min(stride * page, LONGEST)) | (keep & ((table < 0) | (table >= pages))).any(1)
    long = lens + new > min(stride * page, LONGEST)
    fine = ~lost & ~long
    keep &= ~lost[:, None]
    used = torch.zeros(pages + 1, dtype=torch.bool, device=dev)
    used[torch.where(keep, table, pages)] = True
    if s["held"] is not None:
        used[:-1] |= s["held"] != 0
    used[pages] = True
    free = torch.sort(used.to(torch.int8), stable=True)[1]
    # 4: the pages, or the rows, of the requests up to this one are more than there are
    need = torch.where(fine, (lens + new + page - 1) // page - have, 0)
    asked, rows = need.cumsum(0), torch.where(fine, new, 0).cumsum(0)
    served = fine & ((need == 0) | (asked <= (~used).sum())) & ((new == 0) | (rows <= s["rows"]))
    fresh = served[:, None] & (i >= have[:, None]) & (i < (have + need)[:, None])
    nth = ((asked - need - have)[:, None] + i).clamp(0, pages)
    out = torch.where(fresh, free[nth], torch.where(keep, table, -1))
    starts = torch.zeros(seqs + 1, dtype=torch.int64, device=dev)
    starts[1:] = torch.where(served, new, 0).cumsum(0)
    row = torch.arange(s["rows"], device=dev)
    seq = (row[:, None] >= starts[None, 1:]).sum(-1)
    some, seq = seq < seqs, seq.clamp(max=seqs - 1)
    position = lens[seq] + row - starts[seq]
    slot = out[seq, (position // page).clamp(max=stride - 1)] * page + position % page
    status = torch.where(lost, 3, torch.where(long, 7, torch.where(served, 0, 4)))
    length = torch.where(lost, 0, torch.where(served, lens + new, lens))
    return {"table": out.to(torch.int32), "lens": length.to(torch.int32), "starts": starts.to(torch.int32),
            "slots": torch.where(some, slot, -1), "positions": torch.where(some, position, -1).to(torch.int32),
            "status": status.to(torch.int32)}


def _remainder(random, z):
    """random modulo z, random's bits taken as an unsigned number; z below 2^61."""
    half = (random >> 1) & (2**63 - 1)
    return (2 * (half % z) + (random & 1)) % z


def _sample(s):
    logits, dev = s["logits"], s["logits"].device
    rows, vocab = logits.shape
    t = s["temperature"].long()[:, None]
    masked = logits == MIN
    m = logits.amax(-1, keepdim=True)
    low = torch.where(m > MIN + FAR, m - FAR, MIN)
    d = torch.where(masked, 2**63 - 1, m - torch.maximum(logits, low))
    index = torch.where(d >= 16 * t, 4096, (d.clamp(max=2**24) << 8) // t.clamp(min=1))
    e = torch.where(masked, 0, s["exp"].long()[index])
    e = torch.where(t > 0, e, 0)
    # by distance, then by token: what is kept is a beginning of this order
    order = torch.sort(d, dim=-1, stable=True)[1]
    sums = e.gather(1, order)
    most = sums[:, :1] * 1
    count = (~masked).sum(-1)
    n = count if s["top_k"] is None else torch.where(s["top_k"] > 0, torch.minimum(count, s["top_k"].long()), count)
    if s["min_p"] is not None:
        least = s["min_p"].long().clamp(max=ONE)[:, None]
        enough = (((sums << 24) >= least * most).sum(-1)).clamp(min=1)
        enough = torch.minimum(enough, count)
    sums = sums.cumsum(-1)
    last = (n - 1).clamp(min=0)[:, None]
    if s["top_p"] is not None:
        z = sums.gather(1, last)
        p = s["top_p"].long().clamp(max=ONE)[:, None]
        target = (z >> 24) * p + (((z & (2**24 - 1)) * p) >> 24)     # floor(z p / 2^24)
        n = torch.where(p[:, 0] < ONE, torch.minimum(n, (sums < target).sum(-1) + 1), n)
    if s["min_p"] is not None:
        n = torch.minimum(n, enough)
    n = torch.where(t[:, 0] > 0, n, count.clamp(max=1))
    kept = torch.zeros_like(masked).scatter(1, order, torch.arange(vocab, device=dev) < n[:, None])
    weight = torch.where(kept, e, 0)
    walk = weight.cumsum(-1)
    z = walk[:, -1].clamp(min=1)
    r = _remainder(s["random"], z)
    token = torch.where(t[:, 0] > 0, (walk <= r[:, None]).sum(-1), order[:, 0]).clamp(max=vocab - 1)
    prob = (weight.gather(1, token[:, None])[:, 0] << 24) // z
    prob = torch.where(t[:, 0] > 0, prob, ONE)
    some = n > 0
    return {"token": torch.where(some, token, -1).to(torch.int32), "prob": torch.where(some, prob, 0).to(torch.int32),
            "kept": n.to(torch.int32)}


def exact(case, seed):
    """The same from the definitions on the host: numpy on 64-bit words, and Python's integers."""
    import numpy as np
    c = case
    if c["op"] == "window" and 16 * work(c)["flops"] > 3e11:
        return None
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

    if c["op"] == "window":
        hd, group, page = c["head"], c["heads"] // c["kv_heads"], c["page"]
        table = np.array(_exp_table(), dtype=np.int64)
        out = np.zeros((s["rows"], c["heads"] * hd), dtype=np.int64)
        for i, (n, length) in enumerate(zip(_news(c), _lens(c))):
            r0, first = int(h["starts"][i]), length - n
            t = np.array([x for x in range(length) if x < c["sinks"] or x > first - c["window"]], dtype=np.int64)
            pos = (first + np.arange(n))[:, None]
            seen = (t <= pos) & ((t < c["sinks"]) | (pos - t < c["window"]))
            pg, sl = h["table"][i].astype(np.int64)[t // page], t % page
            for head in range(c["heads"]):
                kk, vv = (h[x][pg, 0, head // group, sl].astype(np.int64) for x in "kv")
                q = h["q"][r0:r0 + n, head * hd:(head + 1) * hd]
                score = ((product(q, kk.T.copy()) >> 16) * s["inv"]) >> 24
                m = np.where(seen, score, MIN).max(-1, keepdims=True)
                e = np.where(seen, table[np.minimum((m - np.minimum(score, m)) >> 8, 4096)], 0)
                p = (e << 24) // e.sum(-1, keepdims=True)
                out[r0:r0 + n, head * hd:(head + 1) * hd] = product(p, vv) >> 24
        return {"out": out, "status": h["status"]}
    if c["op"] == "advance":
        page, stride, asks, held = c["page"], h["table"].shape[1], _asks(c), h.get("held")
        most = min(stride * page, LONGEST)
        used, rows = {i for i in range(s["pages"]) if held is not None and held[i]}, []
        for r, (n, ask) in enumerate(zip(_lens(c), asks)):
            mine = {}
            for i in range(-(-min(n, stride * page) // page)):
                # the first position after the sequence's sees the page, or one of the first ones lies in it
                if not c["window"] or i * page < c["sinks"] or n - ((i + 1) * page - 1) < c["window"]:
                    mine[i] = int(h["table"][r, i])
            status = 3 if n > most or any(not 0 <= w < s["pages"] for w in mine.values()) else 7 if n + ask > most else 0
            if status == 3:
                mine, n = {}, 0
            used |= set(mine.values())
            rows.append([mine, n, ask, status])
        free = [w for w in range(s["pages"]) if w not in used]
        taken = asked = granted = 0
        starts, slots, positions = [0], [], []
        for row in rows:
            mine, n, ask, status = row
            if status == 0:
                have = -(-n // page)
                need = -(-(n + ask) // page) - have
                taken, asked = taken + need, asked + ask
                if (need and taken > len(free)) or (ask and asked > s["rows"]):
                    row[3] = 4
                else:
                    mine.update(zip(range(have, have + need), free[taken - need:taken]))
                    row[1], granted = n + ask, granted + ask
                    positions += range(n, n + ask)
                    slots += [mine[p // page] * page + p % page for p in range(n, n + ask)]
            starts.append(granted)
        table = np.full(h["table"].shape, -1, dtype=np.int32)
        for r, row in enumerate(rows):
            for i, w in row[0].items():
                table[r, i] = w
        rest = [-1] * (s["rows"] - granted)
        return {"table": table, "lens": np.array([r[1] for r in rows], dtype=np.int32),
                "starts": np.array(starts, dtype=np.int32), "slots": np.array(slots + rest, dtype=np.int64),
                "positions": np.array(positions + rest, dtype=np.int32),
                "status": np.array([r[3] for r in rows], dtype=np.int32)}
    table, token, prob, count = np.array(_exp_table(), dtype=np.int64), [], [], []
    for r in range(c["rows"]):
        row, t = h["logits"][r], int(h["temperature"][r])
        allowed = np.flatnonzero(row != MIN)
        if not len(allowed):
            token, prob, count = token + [-1], prob + [0], count + [0]
            continue
        d = row[allowed].max() - row[allowed]
        order = np.argsort(d, kind="stable")
        if t == 0:
            token, prob, count = token + [int(allowed[order[0]])], prob + [ONE], count + [1]
            continue
        e = table[np.where(d >= 16 * t, 4096, np.minimum(d, 16 * t) * 256 // t)]
        n = len(allowed)
        if c["k"] and 0 < h["top_k"][r] < n:
            n = int(h["top_k"][r])
        ahead = np.cumsum(e[order])
        if c["p"] and h["top_p"][r] < ONE:
            target = (int(ahead[n - 1]) * int(h["top_p"][r])) >> 24
            n = min(n, 1 + int(np.searchsorted(ahead, target)))
        if c["m"]:
            n = max(1, min(n, int(((e << 24) >= int(h["min_p"][r]) * int(e.max())).sum())))
        keep = np.sort(order[:n])
        walk = np.cumsum(e[keep])
        z = int(walk[-1])
        at = int(np.searchsorted(walk, (int(h["random"][r]) % 2**64) % z, side="right"))
        token.append(int(allowed[keep[at]]))
        prob.append((int(e[keep[at]]) << 24) // z)
        count.append(n)
    return {"token": np.array(token, dtype=np.int32), "prob": np.array(prob, dtype=np.int32),
            "kept": np.array(count, dtype=np.int32)}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"window": _window, "advance": _advance, "sample": _sample}[op](s)
    import fixed_point_int8_gb300 as ck
    if op == "window":
        rc, out = ck.paged_attention(s["cache"], 0, s["batch"], s["q"], s["exp"], s["inv"], out=s["out"],
                                     work=s["work"], window=s["view"])
        result = {"out": out, "status": s["status"]}
    elif op == "advance":
        c = s["case"]
        view = ck.Window(c["sinks"], c["window"]) if c["window"] else None
        rc, got = s["plan"].advance(s["lens"], s["table"], s["new"], s["rows"], window=view, held=s["held"])
        result = {"table": got.table, "lens": got.lens, "starts": got.starts, "slots": got.slots,
                  "positions": got.positions, "status": got.status}
    else:
        rc, got = ck.sample(s["logits"], s["temperature"], s["random"], s["exp"], top_k=s["top_k"], top_p=s["top_p"],
                            min_p=s["min_p"])
        result = {"token": got.token, "prob": got.prob, "kept": got.kept}
    if rc:
        raise RuntimeError("%s: error %d" % (op, rc))
    return result
