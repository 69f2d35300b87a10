"""Workloads of the operators that end and verify a decoding step.

Each case is one pass through one operator at sizes that serving a decoder
meets, speculative decoding with trees of drafted tokens among them:

* ``tree``    attention of drafted tokens over the paged int8 cache: each sees
              the sequence's cached tokens and its own ancestors
* ``sample``  next tokens from logits and given random numbers: temperature,
              top-k, top-p, min-p
* ``keep``    the drafted tokens that the sampled ones confirm, and their keys
              and values moved together in the cache
* ``fork``    pages of the cache shared by sequences that continue another one,
              fresh pages for the next tokens, copies of the pages they write
* ``compact`` the pages in use moved together at the front of the pool

``run`` computes a case in its plain form (elementary torch operations in 32
bits, sampling in 64) or, where ``own`` is true, by the package's own
operators.  Int8 results are returned as the values they stand for.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one sequence's tree of 26 drafted tokens: latency
        {"name": "tree-one", "op": "tree", "batch": 1, "q": 26, "len": 2001, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 64, "window": 0},
        # a server verifies up to 64 drafted tokens for each of 16 sequences
        {"name": "tree-batch", "op": "tree", "batch": 16, "q": 64, "len": 4096, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 64, "window": 0},
        # small trees behind long documents: the cache is read once
        {"name": "tree-long", "op": "tree", "batch": 4, "q": 13, "len": 50000, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 32, "window": 0},
        # wide trees in small pages, heads of 64, a sliding window
        {"name": "tree-wide", "op": "tree", "batch": 6, "q": 200, "len": 1700, "heads": 16, "kv_heads": 4,
         "head_dim": 64, "page": 16, "window": 1024},
        # the next token of one sequence: latency
        {"name": "sample-one", "op": "sample", "rows": 1, "vocab": 32000, "dtype": "fp16", "filters": "k50 p"},
        # a decode step of 64 sequences, nucleus sampling
        {"name": "sample-batch", "op": "sample", "rows": 64, "vocab": 128256, "dtype": "fp16", "filters": "p"},
        # every node of 16 trees, each request with settings of its own
        {"name": "sample-tree", "op": "sample", "rows": 801, "vocab": 152064, "dtype": "fp16",
         "filters": "mixed"},
        # logits that a program has worked on in fp32, an odd vocabulary
        {"name": "sample-wide", "op": "sample", "rows": 33, "vocab": 50257, "dtype": "fp32", "filters": "m"},
        # one sequence's tree of 26 tokens, 4 of them confirmed
        {"name": "keep-one", "op": "keep", "batch": 1, "q": 26, "len": 1000, "deep": 4, "kv_heads": 8,
         "head_dim": 128, "page": 64},
        # 96 trees of up to 64 tokens in small pages, up to 9 confirmed
        {"name": "keep-batch", "op": "keep", "batch": 96, "q": 64, "len": 300, "deep": 9, "kv_heads": 8,
         "head_dim": 128, "page": 16},
        # a step of beam search: 16 requests of 4 beams
        {"name": "fork-beams", "op": "fork", "groups": 16, "beams": 4, "len": 500, "tokens": 1, "kv_heads": 8,
         "head_dim": 128, "page": 16},
        # a pool of 1500 pages half in use after many requests have ended
        {"name": "compact-pool", "op": "compact", "pages": 1500, "batch": 40, "live": 0.5, "kv_heads": 4,
         "head_dim": 128, "page": 64},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "sample", "sample", "sample", "keep", "fork", "compact"])
    if op == "sample":
        rows = _spread(rng, 1, 801)
        vocab = _spread(rng, 1000, min(262144, 801 * 152064 // rows))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(["fp16", "fp16", "fp32"]),
                "filters": rng.choice(["", "k50", "k50 p", "p", "m", "p m", "k1000", "mixed"])}
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        heads, kv_heads = rng.choice([(32, 8), (64, 8), (32, 32), (16, 2), (12, 4), (28, 4)])
        dim = rng.choice([64, 128, 128, 128, 256])
        q = _spread(rng, 2, 200)
        batch = _spread(rng, 1, max(1, min(32, 2 ** 22 // (heads * dim * q))))
        room = min(2 ** 27 // (batch * kv_heads * dim), 2 ** 34 // (batch * heads * q * dim))
        return {"op": op, "batch": batch, "q": q, "len": _spread(rng, q, max(q, min(50000, room))), "heads": heads,
                "kv_heads": kv_heads, "head_dim": dim, "page": page,
                "window": rng.choice([0, 0, 0, _spread(rng, 64, 4096)])}
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    shape = {"op": op, "kv_heads": kv_heads, "head_dim": dim, "page": page}
    if op == "keep":
        q = _spread(rng, 2, 128)
        room = min(1000, 2 ** 26 // (kv_heads * dim * 96))
        return {**shape, "batch": _spread(rng, 1, 96), "q": q, "len": _spread(rng, q, max(q, room)),
                "deep": rng.randint(1, min(q, 12))}
    if op == "fork":
        return {**shape, "groups": _spread(rng, 1, 32), "beams": rng.randint(1, 8), "tokens": _spread(rng, 1, 2 * page),
                "len": _spread(rng, 1, min(600, 2 ** 27 // (kv_heads * dim * 256)))}
    return {**shape, "pages": _spread(rng, 50, min(4000, 2 ** 27 // (2 * kv_heads * page * dim))),
            "batch": _spread(rng, 1, 64), "live": rng.uniform(0.1, 0.9)}


def _spans(case):
    """(tokens a sequence holds in all, drafted tokens among them, confirmed
    ones), for each sequence; fixed by the case alone, so that work() knows."""
    rng = random.Random(case["batch"] * 1000003 + case["len"] * 1009 + case["q"])
    spans = []
    for b in range(case["batch"]):
        new = case["q"] if b == 0 else rng.randint(max(1, case["q"] // 4), case["q"])
        total = case["len"] if b == 0 else rng.randint(max(new, case["len"] // 4), max(new, case["len"]))
        most = min(case.get("deep", 1), new)
        spans.append((max(total, new), new, most if b == 0 else rng.randint(1, most)))
    return spans


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    state = dict(case)
    {"tree": _trees, "keep": _trees, "sample": _logits, "fork": _beams, "compact": _pool}[case["op"]](state, gen, rng)
    return state


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _cache(s, gen, pages):
    """A paged int8 cache of normal values."""
    s["kv_cache"] = torch.empty(pages, 2, s["kv_heads"], s["page"], s["head_dim"], dtype=torch.int8, device="cuda")
    step = max(1, (1 << 27) // s["kv_cache"][0].numel())
    for at in range(0, pages, step):
        part = s["kv_cache"][at:at + step]
        part.copy_((34 * _normal(gen, *part.shape)).round_().clamp_(-127, 127))
    size = 0.6 + 0.8 * torch.rand(pages, 2, s["kv_heads"], generator=gen, device="cuda")
    s["kv_scale"] = (size / 34).half()


def _trees(s, gen, rng):
    """Sequences over a shuffled pool, the last tokens of each a tree of drafted
    ones: parents before children, node 0 the root."""
    spans = _spans(s)
    used = [-(-length // s["page"]) for length, _, _ in spans]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    place = torch.zeros(s["batch"], max(used), dtype=torch.int64)
    done = 0
    for b, n in enumerate(used):
        place[b, :n] = torch.arange(done, done + n)
        done += n
    ends, parents, drafted, sampled = [0], [], [], []
    for _, new, deep in spans:
        # a path of `deep` nodes is confirmed; the others hang anywhere, near
        # the root more often
        path = [0] + sorted(rng.sample(range(1, new), deep - 1))
        follow = dict(zip(path, path[1:]))
        before = {c: p for p, c in follow.items()}
        token = rng.sample(range(32000), new)
        ends.append(ends[-1] + new)
        parents += [-1] + [before.get(i, int(i * rng.random() ** 1.5)) for i in range(1, new)]
        drafted += token
        sampled += [token[follow[i]] if i in follow else 32000 + rng.randrange(100) for i in range(new)]
    put = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    s["block_table"] = order[place.cuda()]
    s["seq_lens"], s["cu_q"] = put([length for length, _, _ in spans]), put(ends)
    s["max_len"] = max(length for length, _, _ in spans)
    s["parents"], s["drafted"], s["sampled"] = put(parents), put(drafted), put(sampled)
    _cache(s, gen, pages)
    if s["op"] == "tree":
        s["queries"] = (2 * _normal(gen, ends[-1], s["heads"], s["head_dim"])).half()
        s["scale"] = s["head_dim"] ** -0.5
        # which of its sequence's drafted tokens a node sees, a bit each
        words = -(-s["q"] // 32)
        mask = torch.zeros(ends[-1], 32 * words, dtype=torch.bool)
        at = 0
        for lo, hi in zip(ends, ends[1:]):
            for i in range(hi - lo):
                if parents[at] >= 0:
                    mask[at] = mask[lo + parents[at]]
                mask[at, i] = True
                at += 1
        bits = (mask.view(-1, words, 32).long() << torch.arange(32)).sum(dim=2)
        s["mask"] = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).cuda()


def _logits(s, gen, rng):
    """Rows of normal logits with a few that stand out."""
    rows, vocab = s["rows"], s["vocab"]
    x = 2.2 * _normal(gen, rows, vocab)
    high = torch.randint(vocab, (rows, 20), generator=gen, device="cuda")
    x.scatter_add_(1, high, 7 - 2.5 * torch.rand(rows, 20, generator=gen, device="cuda").clamp_(min=1e-6).log_())
    s["logits"] = x.half() if s["dtype"] == "fp16" else x
    s["u"] = torch.rand(rows, generator=gen, device="cuda")
    if s["filters"] == "mixed":        # settings of each row's request
        pick = lambda values, dtype: torch.tensor([rng.choice(values) for _ in range(rows)], dtype=dtype).cuda()
        s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.3], torch.float32)
        s["top_k"] = pick([0, 0, 20, 50, 400], torch.int32)
        s["top_p"] = pick([1.0, 0.9, 0.95], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.05], torch.float32)
        return
    s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.8, 0, 1.0, 0.0
    for name in s["filters"].split():
        if name[0] == "k":
            s["top_k"] = int(name[1:])
        else:
            s.update({"top_p": 0.9} if name == "p" else {"min_p": 0.05})


def _beams(s, gen, rng):
    """Groups of beams: a group's sequences are of one length and share all
    pages but their last few; the next step continues some of them twice."""
    page, beams = s["page"], s["beams"]
    table, lens, parent, pages = [], [], [], 0
    fixed = random.Random(s["len"] * 1009 + s["groups"] * 31 + beams)    # the pool's size is the case's
    for g in range(s["groups"]):
        length = s["len"] if g == 0 else fixed.randint(max(1, s["len"] // 4), s["len"])
        used = -(-length // page)
        shared = max(0, used - fixed.randint(1, 3))
        first = list(range(pages, pages + shared))
        pages += shared
        for _ in range(beams):
            table.append(first + list(range(pages, pages + used - shared)))
            pages += used - shared
            lens.append(length)
            parent.append(beams * g + rng.randrange(beams))
    room = -(-(s["len"] + s["tokens"]) // page)
    fresh = sum(-(-(n + s["tokens"]) // page) - n // page for n in lens)
    s["pages"] = pages + fresh + 5
    order = torch.randperm(s["pages"], generator=gen, device="cuda").to(torch.int32)
    place = torch.full((len(table), room), -1, dtype=torch.int64)
    refs = torch.zeros(s["pages"], dtype=torch.int32)
    for b, row in enumerate(table):
        place[b, :len(row)] = torch.tensor(row)
        for p in row:
            refs[p] += 1
    place = place.cuda()
    s["block_table"] = torch.where(place >= 0, order[place.clamp(min=0)], -1)
    s["refs"] = torch.zeros_like(order).scatter_(0, order.long(), refs.cuda())
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["parent"] = torch.tensor(parent, dtype=torch.int32).cuda()
    _cache(s, gen, s["pages"])


def _pool(s, gen, rng):
    """A pool with pages in use here and there, some by two sequences."""
    live = max(1, min(s["pages"] - 1, round(s["pages"] * s["live"])))
    order = torch.randperm(s["pages"], generator=gen, device="cuda")[:live].cpu()
    rows = [[] for _ in range(s["batch"])]
    shares = [rng.uniform(0.5, 1.0) for _ in rows]
    at, total = 0.0, sum(shares)
    for row, share in zip(rows, shares):
        row += order[round(at * live):round((at + share / total) * live)].tolist()
        at += share / total
    for b in range(1, len(rows), 5):
        rows[b] = rows[b - 1][:len(rows[b - 1]) // 2] + rows[b]
    table = torch.full((len(rows), 3 * live // len(rows) + 40), -1, dtype=torch.int32)
    for b, r in enumerate(rows):
        table[b, :len(r)] = torch.tensor(r, dtype=torch.int32)
    s["refs"] = torch.bincount(table[table >= 0].long(), minlength=s["pages"]).to(torch.int32).cuda()
    s["block_table"] = table.cuda()
    _cache(s, gen, s["pages"])


# --------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


def _run_own(s):
    import w4a8_gemm_amd as w4
    if s["op"] == "tree":
        return {"o": w4.tree_attention(s["queries"], s["kv_cache"], s["kv_scale"], s["block_table"], s["seq_lens"],
                                       s["mask"], cu_q=s["cu_q"], max_q=s["q"], max_len=s["max_len"],
                                       scale=s["scale"], window=s["window"])}
    if s["op"] == "sample":
        tokens, probs = w4.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
        return {"tokens": tokens, "probs": probs}
    cache, scale = s["kv_cache"], s["kv_scale"]
    if s["op"] == "keep":
        path, count, tokens, lens = w4.tree_accept(s["drafted"], s["parents"], s["sampled"], s["seq_lens"],
                                                   cu_q=s["cu_q"], max_q=s["q"])
        w4.kv_keep(cache, scale, s["block_table"], s["seq_lens"], path, count, cu_q=s["cu_q"])
        return {"path": path, "count": count, "tokens": tokens, "lens": lens,
                "kv": cache * scale[..., None, None]}
    if s["op"] == "fork":
        table, lens, refs = w4.kv_fork(s["block_table"], s["seq_lens"], s["refs"], s["parent"], s["page"])
        table, lens, refs, src, dst, counts = w4.kv_alloc(table, lens, refs, s["tokens"], s["page"])
    else:
        table, refs, place, src, dst, counts = w4.kv_compact(s["block_table"], s["refs"])
        lens = place
    w4.kv_copy_pages(cache, scale, src, dst, counts)
    return {"table": table, "lens": lens, "refs": refs, "counts": counts, "kv": cache * scale[..., None, None]}


def _plain_tree(s):
    heads, kv_heads, dim, page = s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    cu, lens, table = s["cu_q"].long(), s["seq_lens"].long(), s["block_table"].long()
    batch, most, length, group = s["batch"], s["q"], table.shape[1] * page, heads // kv_heads
    total = s["queries"].shape[0]

    def gathered(which):   # [batch, kv_heads, length, dim]
        values = s["kv_cache"][:, which][table] * s["kv_scale"][:, which][table].float()[..., None, None]
        return values.transpose(1, 2).reshape(batch, kv_heads, length, dim)

    # queries padded to [batch, kv_heads, group * most, dim]
    new = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + torch.arange(most, device=cu.device)).clamp(max=total - 1)
    padded = s["queries"][rows].float().view(batch, most, kv_heads, group, dim).permute(0, 2, 3, 1, 4)
    padded = padded.reshape(batch, kv_heads, group * most, dim)
    scores = torch.matmul(padded, gathered(0).transpose(2, 3).contiguous()).mul_(s["scale"])

    # cached tokens, then the drafted ones that the mask names
    key = torch.arange(length, device=cu.device)
    node = key - (lens - new)[:, None]                          # [batch, length]
    words = s["mask"][rows]                                     # [batch, most, words]
    at = node.clamp(min=0, max=32 * words.shape[2] - 1)[:, None].expand(batch, most, length)
    bits = (words.gather(2, at // 32) >> (at % 32)) & 1
    seen = torch.where((node >= 0)[:, None], bits == 1, True) & (key < lens[:, None])[:, None]
    if s["window"]:                                             # the last ones of all that a node sees
        seen &= seen.long().flip(2).cumsum(2).flip(2) <= s["window"]
    scores = scores.view(batch, kv_heads, group, most, length)
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    scores.sub_(scores.amax(dim=-1, keepdim=True).clamp_(min=-1e30)).exp_()
    weight = scores.sum(dim=-1, keepdim=True)
    out = torch.matmul(scores.view(batch, kv_heads, group * most, length), gathered(1))
    out = out.view(batch, kv_heads, group, most, dim) / torch.where(weight > 0, weight, 1.0)
    # back to one row per token
    token = torch.arange(total, device=cu.device)
    seq = torch.bucketize(token, cu[1:], right=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch * most, heads, dim)
    return {"o": out[seq * most + token - cu[seq]].half()}


def _plain_sample(s):
    x = s["logits"]
    rows, vocab = x.shape

    def column(name):
        v = s[name]
        return v.double()[:, None] if torch.is_tensor(v) else torch.full((rows, 1), v, dtype=torch.float64, device=x.device)
    temperature, top_k, top_p, min_p = map(column, ("temperature", "top_k", "top_p", "min_p"))
    value, order = torch.sort(x, dim=1, descending=True, stable=True)
    value = value.double()
    weight = torch.exp((value - value[:, :1]) / torch.where(temperature > 0, temperature, 1.0))
    rank = torch.arange(vocab, device=x.device)
    keep = (rank < torch.where(top_k > 0, top_k, vocab)) & ((temperature > 0) | (rank < 1))
    weight = torch.where(keep, weight, 0.0)
    upto = weight.cumsum(dim=1)
    keep = (upto - weight < top_p * upto[:, -1:]) | (top_p >= 1)
    keep &= weight >= min_p
    # drawn in the vocabulary's order
    upto = torch.zeros_like(weight).scatter_(1, order, torch.where(keep, weight, 0.0)).cumsum(dim=1)
    token = (upto <= s["u"].double()[:, None] * upto[:, -1:]).sum(dim=1, keepdim=True)
    mass = torch.exp((x.gather(1, token).double() - value[:, :1]) / torch.where(temperature > 0, temperature, 1.0))
    return {"tokens": token[:, 0].to(torch.int32), "probs": (mass / upto[:, -1:])[:, 0].float()}


def _plain_keep(s):
    cu, lens, table, page, batch = s["cu_q"].long(), s["seq_lens"].long(), s["block_table"].long(), s["page"], s["batch"]
    dev, most = cu.device, s["q"]
    total = s["parents"].shape[0]
    node = torch.arange(total, device=dev)
    seq = torch.bucketize(node, cu[1:], right=True)
    # from each root to the child that holds the token sampled there
    current = torch.zeros(batch, dtype=torch.int64, device=dev)
    going = torch.ones(batch, dtype=torch.bool, device=dev)
    path = torch.full((batch, most), -1, dtype=torch.int64, device=dev)
    path[:, 0] = 0
    last = cu[:-1].clone()
    for step in range(1, most):
        fits = (s["parents"] == current[seq]) & (s["drafted"] == s["sampled"][last][seq]) & going[seq]
        child = torch.where(fits, node - cu[seq], total)
        child = torch.full((batch,), total, device=dev).index_reduce_(0, seq, child, "amin")
        going = child < total
        current = torch.where(going, child, current)
        path[:, step] = torch.where(going, child, -1)
        last = cu[:-1] + current
    count = (path >= 0).sum(dim=1)
    tokens = s["sampled"][last]

    # their keys and values, behind the sequence's cached tokens
    start = lens - (cu[1:] - cu[:-1])
    moved = path >= 0
    owner = torch.arange(batch, device=dev)[:, None].expand_as(path)[moved]
    take = (start[:, None] + path)[moved]
    put = (start[:, None] + torch.arange(most, device=dev))[moved]
    source, target = table[owner, take // page], table[owner, put // page]
    cache, scale = s["kv_cache"], s["kv_scale"].float()
    # a written page's scale: the largest of what it holds then
    after = torch.zeros_like(scale)
    after.index_reduce_(0, target, scale[source], "amax")
    held = table[torch.arange(batch, device=dev), (start // page).clamp(max=table.shape[1] - 1)]
    partly = start % page > 0
    after.index_reduce_(0, held, torch.where(partly[:, None, None], scale[held], 0.0), "amax")
    written = torch.zeros(cache.shape[0], dtype=torch.bool, device=dev).index_fill_(0, target, True)[:, None, None]
    after = torch.where(written, after, scale)
    ratio = lambda old, new: torch.where(old == new, 1.0, old / torch.where(new > 0, new, 1.0))[..., None]
    codes = cache[source, :, :, take % page].float()
    codes = (codes * ratio(scale[source], after[target])).round_()
    filled = torch.zeros(cache.shape[0], dtype=torch.int64, device=dev)
    filled[held] = start % page                               # slots with earlier tokens
    old = (torch.arange(page, device=dev) < filled[:, None])[:, None, None, :, None]
    turned = torch.where(old, (cache * ratio(scale, after)[..., None]).round_().to(torch.int8), cache)
    turned[target, :, :, put % page] = codes.to(torch.int8)
    cache.copy_(turned)
    s["kv_scale"].copy_(after)
    return {"path": path.to(torch.int32), "count": count.to(torch.int32), "tokens": tokens,
            "lens": (start + count).to(torch.int32), "kv": cache * s["kv_scale"][..., None, None]}


def _counts_of(table, pages):
    """How often the entries of a table name each page."""
    flat = torch.where(table >= 0, table, pages).flatten().long()
    return torch.zeros(pages + 1, dtype=torch.int32, device=table.device).index_add_(
        0, flat, torch.ones_like(flat, dtype=torch.int32))[:pages]


def _copied(s, source, target, count):
    """The first `count` pairs of pages copied."""
    valid = torch.arange(source.shape[0], device=source.device) < count
    move = torch.arange(s["kv_cache"].shape[0], device=source.device)
    spare = move.shape[0]
    move = torch.cat([move, move[:1]]).scatter_(0, torch.where(valid, target, spare).long(), source.long())[:spare]
    s["kv_cache"].copy_(s["kv_cache"][move])
    s["kv_scale"].copy_(s["kv_scale"][move])
    return s["kv_cache"] * s["kv_scale"][..., None, None]


def _plain_fork(s):
    page, pages, parent = s["page"], s["pages"], s["parent"].long()
    row = torch.arange(parent.shape[0], device=parent.device)
    column = torch.arange(s["block_table"].shape[1], device=parent.device)
    # a row continues its parent: all of its pages, or those with tokens of another
    lens = s["seq_lens"][parent]
    used = (lens + page - 1) // page
    shared = (column < used[:, None]) | (parent == row)[:, None]
    table = torch.where(shared, s["block_table"][parent], -1)
    refs = s["refs"] - _counts_of(s["block_table"], pages) + _counts_of(table, pages)
    # pages for the next tokens: entries without one, and shared pages that get them
    end = lens + s["tokens"]
    first = lens // page
    wanted = (column >= first[:, None]) & (column < ((end + page - 1) // page)[:, None])
    half = (column == first[:, None]) & (lens % page > 0)[:, None] & wanted
    held = torch.where(half & (table >= 0), table, pages).long()        # pages under copy, if shared
    writers = torch.zeros(pages + 1, dtype=torch.int32, device=parent.device)
    writers.index_add_(0, held.flatten(), torch.ones_like(held.flatten(), dtype=torch.int32))
    final = torch.full((pages + 1,), -1, device=parent.device)
    final.index_reduce_(0, held.flatten(), row[:, None].expand_as(held).flatten(), "amax")
    owners = torch.cat([refs, refs[:1]])
    # the last of a page's holders keeps it, if all of them write
    keeps = (writers[held] >= owners[held]) & (final[held] == row[:, None])
    copies = (held < pages) & (owners[held] > 1) & ~keeps
    wants = (wanted & (table < 0)) | copies
    number = wants.flatten().long().cumsum(0).view_as(wants) - 1
    free = refs <= 0
    place = torch.where(free, free.long().cumsum(0) - 1, pages)
    by_number = torch.full((pages + 1,), -1, device=parent.device)
    by_number.scatter_(0, place, torch.arange(pages, device=parent.device))
    fresh = torch.where(number < pages, by_number[number.clamp(min=0, max=pages - 1)], -1).to(torch.int32)
    missing = (wants.sum() - free.sum()).clamp(min=0)
    handed = torch.where(wants, fresh, -1)
    refs = refs - torch.zeros_like(writers).index_add_(0, torch.where(copies, table, pages).flatten().long(),
                                                       torch.ones_like(table.flatten()))[:pages] \
        + _counts_of(handed, pages)
    copied = copies & (handed >= 0)
    pairs, each = copied.sum(), torch.arange(copies.numel(), device=parent.device).view_as(copies)
    at = torch.where(copied, each, copies.numel() - 1).flatten().sort().values[:parent.shape[0]]
    kv = _copied(s, table.flatten()[at], handed.flatten()[at], pairs)
    table = torch.where(wants, handed, table)
    return {"table": table, "lens": end, "refs": refs, "counts": torch.stack([pairs, missing]).to(torch.int32), "kv": kv}


def _plain_compact(s):
    refs = s["refs"]
    pages = refs.shape[0]
    page = torch.arange(pages, device=refs.device)
    live = (refs > 0).sum()
    # the n-th page in use from `live` on goes to the n-th free one before it
    gap, far = (refs <= 0) & (page < live), (refs > 0) & (page >= live)
    count = far.sum()
    target = torch.where(gap, page, pages).sort().values[:(pages + 1) // 2]
    source = torch.where(far, page, pages).sort().values[:(pages + 1) // 2]
    valid = source < pages
    place = torch.cat([page, page[:1]]).scatter_(0, source, target)[:pages]
    refs = torch.cat([refs, refs[:1]])
    moved = torch.cat([refs[:pages], refs[:1]]).scatter_(0, target, refs[source])
    moved = torch.where(page < live, moved[:pages], 0)
    table = torch.where(s["block_table"] >= 0, place[s["block_table"].clamp(min=0).long()], -1)
    kv = _copied(s, torch.where(valid, source, 0), torch.where(valid, target, 0), count)
    return {"table": table.to(torch.int32), "lens": place.to(torch.int32), "refs": moved.to(torch.int32),
            "counts": torch.stack([count, torch.zeros_like(count)]).to(torch.int32), "kv": kv}


_PLAIN = {"tree": _plain_tree, "sample": _plain_sample, "keep": _plain_keep, "fork": _plain_fork, "compact": _plain_compact}


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "sample":    # every logit read: compared, scaled, its weight taken and added
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "fp16" else 4) + 12 * case["rows"], "flops": 5 * n}
    slot = 2 * case["kv_heads"] * case["head_dim"]            # bytes of a token in the cache
    if case["op"] == "fork":      # tables and counts, a copied page for about half of the rows
        rows = case["groups"] * case["beams"]
        room = -(-(case["len"] + case["tokens"]) // case["page"])
        return {"bytes": rows * room * 8 + rows * 16 + rows // 2 * 2 * case["page"] * slot, "flops": rows * room}
    if case["op"] == "compact":      # about live * (1 - live) of the pages move
        moves = case["pages"] * case["live"] * (1 - case["live"])
        return {"bytes": int(moves * 2 * case["page"] * slot + case["pages"] * 16), "flops": case["pages"]}
    spans = _spans(case)
    total = sum(new for _, new, _ in spans)
    if case["op"] == "keep":
        return {"bytes": 12 * total + sum(2 * slot * deep for _, _, deep in spans), "flops": total}
    heads, dim, window = case["heads"], case["head_dim"], case["window"] or 1 << 40
    read = sum(min(length, window - 1 + new) for length, new, _ in spans)
    pairs = sum(min(length - new, window - 1) * new + new for length, new, _ in spans)
    own_rows = total * (heads * dim * 4 + 4 * -(-case["q"] // 32))
    return {"bytes": read * (slot + 4 * case["kv_heads"] / case["page"]) + own_rows,
            "flops": 4 * heads * dim * pairs}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, sequence by
    sequence, row by row and page by page."""
    s = prepare(case, seed)
    return {"tree": _exact_tree, "sample": _exact_sample, "keep": _exact_keep, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](s)


def _exact_tree(s):
    heads, kv_heads, dim, page, window = s["heads"], s["kv_heads"], s["head_dim"], s["page"], s["window"]
    out = torch.zeros(s["queries"].shape, dtype=torch.float64, device="cuda")
    ends, lens, parents = s["cu_q"].tolist(), s["seq_lens"].tolist(), s["parents"].tolist()
    group = heads // kv_heads
    for b in range(s["batch"]):
        lo, hi, length = ends[b], ends[b + 1], lens[b]
        start = length - (hi - lo)
        hidden = torch.ones(hi - lo, length, dtype=torch.bool)
        for i in range(hi - lo):
            up, line = i, []
            while up >= 0:
                line.append(start + up)
                up = parents[lo + up]
            line = (list(range(start)) + line[::-1])[-window if window else 0:]
            hidden[i, line] = False
        hidden = hidden.cuda()
        at = s["block_table"][b, :-(-length // page)].long()
        for head in range(kv_heads):
            code = s["kv_cache"][at, :, head].double() * s["kv_scale"][at, :, head].double()[..., None, None]
            key, value = code[:, 0].reshape(-1, dim)[:length], code[:, 1].reshape(-1, dim)[:length]
            for g in range(head * group, (head + 1) * group):
                score = s["queries"][lo:hi, g].double() @ key.t().contiguous() * s["scale"]
                score[hidden] = float("-inf")
                out[lo:hi, g] = torch.softmax(score, dim=1) @ value
    return {"o": out}


def _exact_sample(s):
    x, rows = s["logits"], s["rows"]
    cpu = {n: s[n].tolist() if torch.is_tensor(s[n]) else [s[n]] * rows
           for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    tokens, probs = [], []
    for r in range(rows):
        row = x[r].double()
        top = row.max()
        if cpu["temperature"][r] == 0:
            tokens.append(torch.nonzero(row == top)[0, 0])
            probs.append(torch.ones((), dtype=torch.float64, device=row.device))
            continue
        # ids in the order of falling logits, equal ones by their number
        ids = torch.argsort(-row, stable=True)
        if cpu["top_k"][r] > 0:
            ids = ids[:int(cpu["top_k"][r])]
        mass = ((row[ids] - top) / cpu["temperature"][r]).exp()
        n = ids.shape[0]
        if cpu["top_p"][r] < 1:            # the fewest whose mass reaches the share
            n = torch.searchsorted(mass.cumsum(0), cpu["top_p"][r] * mass.sum()) + 1
        few = torch.minimum((mass >= cpu["min_p"][r]).sum(), torch.as_tensor(n, device=row.device))
        chosen = torch.sort(torch.where(torch.arange(ids.shape[0], device=row.device) < few, ids, row.shape[0])).values
        line = torch.cat([row, torch.full_like(row[:1], float("-inf"))])[chosen]
        part = ((line - top) / cpu["temperature"][r]).exp()
        upto = part.cumsum(0)
        at = torch.searchsorted(upto, cpu["u"][r] * upto[-1:], right=True)[0].clamp(max=few - 1)
        tokens.append(chosen[at])
        probs.append(part[at] / upto[-1])
    return {"tokens": torch.stack(tokens).to(torch.int32), "probs": torch.stack(probs)}


def _exact_codes(values, scale):
    """round(values / scale) (64 bits), 0 under a zero scale."""
    return torch.where(scale > 0, torch.round(values / torch.where(scale > 0, scale, 1.0)), 0.0)


def _exact_keep(s):
    page = s["page"]
    codes, scales = s["kv_cache"].double(), s["kv_scale"].double()
    ends, lens, table = s["cu_q"].tolist(), s["seq_lens"].tolist(), s["block_table"].tolist()
    parents, drafted, sampled = s["parents"].tolist(), s["drafted"].tolist(), s["sampled"].tolist()
    paths, tokens, after = [], [], []
    for b in range(s["batch"]):
        lo, hi = ends[b], ends[b + 1]
        path = [0]
        while True:
            fits = [c for c in range(hi - lo) if parents[lo + c] == path[-1] and drafted[lo + c] == sampled[lo + path[-1]]]
            if not fits:
                break
            path.append(fits[0])
        paths.append(path)
        tokens.append(sampled[lo + path[-1]])
        start = lens[b] - (hi - lo)
        after.append(start + len(path))
        values = []
        for node in path:
            at = table[b][(start + node) // page]
            values.append((at, codes[at, :, :, (start + node) % page] * scales[at][..., None]))
        were = scales.clone()
        for index in range(start // page, (start + len(path) - 1) // page + 1):
            at, first = table[b][index], max(0, start - index * page)
            inside = [i for i in range(len(path)) if (start + i) // page == index]
            scale = torch.stack([were[values[i][0]] for i in inside] + ([were[at]] if first else [])).amax(0)
            if first:
                held = codes[at, :, :, :first] * were[at][..., None, None]
                codes[at, :, :, :first] = _exact_codes(held, scale[..., None, None])
            scales[at] = scale
            for i in inside:
                codes[at, :, :, (start + i) % page] = _exact_codes(values[i][1], scale[..., None])
    wide = torch.full((s["batch"], s["q"]), -1, dtype=torch.int32)
    for b, path in enumerate(paths):
        wide[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
    whole = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    return {"path": wide.cuda(), "count": whole([len(p) for p in paths]), "tokens": whole(tokens), "lens": whole(after),
            "kv": codes * scales[..., None, None]}


def _exact_copies(s, pairs):
    cache, scale = s["kv_cache"].clone(), s["kv_scale"].clone()
    for source, target in pairs:
        cache[target], scale[target] = s["kv_cache"][source], s["kv_scale"][source]
    return cache.double() * scale.double()[..., None, None]


def _exact_fork(s):
    page = s["page"]
    old, lens, refs = s["block_table"].tolist(), s["seq_lens"].tolist(), s["refs"].tolist()
    parent = s["parent"].tolist()
    table = [[p if i == j or c < -(-lens[j] // page) else -1 for c, p in enumerate(old[j])] for i, j in enumerate(parent)]
    lens = [lens[j] for j in parent]
    for rows, sign in ((old, -1), (table, 1)):
        for line in rows:
            for p in line:
                if p >= 0:
                    refs[p] += sign
    free = [p for p, n in enumerate(refs) if n <= 0]
    pairs, missing, fixed = [], 0, list(refs)
    ends = [n + s["tokens"] for n in lens]
    before = [list(line) for line in table]
    for b, line in enumerate(table):
        for c in range(lens[b] // page, -(-ends[b] // page)):
            p = before[b][c]
            if p >= 0:
                if c > lens[b] // page or lens[b] % page == 0 or fixed[p] < 2:
                    continue
                holders = [r for r in range(len(before)) if lens[r] % page and before[r][lens[r] // page] == p]
                if len(holders) >= fixed[p] and holders[-1] == b:
                    continue
                refs[p] -= 1
            line[c] = free.pop(0) if free else -1
            missing += line[c] < 0
            if line[c] >= 0:
                refs[line[c]] += 1
                if p >= 0:
                    pairs.append((p, line[c]))
    whole = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    return {"table": whole(table), "lens": whole(ends), "refs": whole(refs), "counts": whole([len(pairs), missing]),
            "kv": _exact_copies(s, pairs)}


def _exact_compact(s):
    refs, table = s["refs"].tolist(), s["block_table"].tolist()
    live = sum(n > 0 for n in refs)
    pairs = list(zip([p for p in range(live, len(refs)) if refs[p] > 0], [p for p in range(live) if refs[p] <= 0]))
    place = list(range(len(refs)))
    for source, target in pairs:
        place[source] = target
        refs[target], refs[source] = refs[source], 0
    whole = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    return {"table": whole([[place[p] if p >= 0 else -1 for p in line] for line in table]), "lens": whole(place),
            "refs": whole(refs), "counts": whole([len(pairs), 0]), "kv": _exact_copies(s, pairs)}
