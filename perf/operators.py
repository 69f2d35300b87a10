"""Workloads of the decoder-layer operators around the W4A8 linear layers.

Each case is one call of one operator at sizes that serving a decoder meets:

* ``norm``       residual addition, root-mean-square norm, per-token int8
* ``swiglu``     silu(gate) * up, per-token int8 (the down projection's input)
* ``append``     rotary positions on queries and keys, keys and values written
                 to a paged int8 cache with one fp16 scale per page and head
* ``attention``  attention that reads that cache, one query token or many

``run`` computes a case in its plain form (elementary torch operations in
fp32, rounded once at the end) or, where ``own`` is true, by the package's own
operators.  Int8 results are returned as the values they stand for.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of a small batch on 4096-wide rows: latency
        {"name": "norm-decode", "op": "norm", "m": 8, "k": 4096},
        # a prefill chunk on 8192-wide rows: bandwidth
        {"name": "norm-prefill", "op": "norm", "m": 4096, "k": 8192},
        # MLP activations of a 13-token decode step (14336 columns)
        {"name": "swiglu-decode", "op": "swiglu", "m": 13, "k": 14336},
        # MLP activations of a prefill chunk (24576 columns)
        {"name": "swiglu-prefill", "op": "swiglu", "m": 2048, "k": 24576},
        # one new token for each of 64 sequences, small pages
        {"name": "append-decode", "op": "append", "batch": 64, "q": 1, "len": 32, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 16, "rotary": 128, "interleaved": False},
        # four prompts of up to 1500 tokens, the first half of each head
        # rotated in adjacent pairs
        {"name": "append-prefill", "op": "append", "batch": 4, "q": 1500, "len": 1700, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "rotary": 64, "interleaved": True},
        # one sequence's next token after 2000 others: latency
        {"name": "attend-one", "op": "attention", "batch": 1, "q": 1, "len": 2001, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "window": 0},
        # the decode step of a busy server: 64 ragged sequences
        {"name": "attend-batch", "op": "attention", "batch": 64, "q": 1, "len": 8192, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "window": 0},
        # the same for a model whose heads do not share keys, small pages
        {"name": "attend-heads", "op": "attention", "batch": 16, "q": 1, "len": 4000, "heads": 64,
         "kv_heads": 64, "head_dim": 128, "page": 16, "window": 0},
        # two very long documents, one token each
        {"name": "attend-long", "op": "attention", "batch": 2, "q": 1, "len": 131072, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 128, "window": 0},
        # chunks of 1 to 200 tokens in one batch, a sliding window of 1024
        {"name": "attend-chunks", "op": "attention", "batch": 12, "q": 200, "len": 4096, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 32, "window": 1024},
        # a prompt of 8192 tokens, read back through the cache
        {"name": "attend-prompt", "op": "attention", "batch": 1, "q": 8192, "len": 8192, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "page": 64, "window": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "swiglu", "append", "attention", "attention"])
    if op == "norm":
        k = 128 * _spread(rng, 8, 64)
        return {"op": op, "m": _spread(rng, 1, 4096), "k": k}
    if op == "swiglu":
        k = 128 * _spread(rng, 16, 192)
        return {"op": op, "m": _spread(rng, 1, 2048), "k": k}
    heads, kv_heads = rng.choice([(32, 8), (64, 8), (32, 32), (64, 64), (16, 2), (12, 4), (28, 4)])
    head_dim = rng.choice([64, 128, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        rotary = rng.choice([head_dim, head_dim, head_dim // 2])
        shape = {"op": op, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
                 "rotary": rotary, "interleaved": rng.random() < 0.5}
        if rng.random() < 0.5:
            return {**shape, "batch": _spread(rng, 1, 128), "q": 1, "len": _spread(rng, 2, 2 * page)}
        q = _spread(rng, 2, 1500)
        return {**shape, "batch": _spread(rng, 1, max(1, min(16, 4500 // q))), "q": q,
                "len": q + rng.randrange(200)}
    shape = {"op": op, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
             "window": rng.choice([0, 0, 0, _spread(rng, 64, 4096)])}
    if rng.random() < 0.6:
        batch = _spread(rng, 1, 64)
        room = 2 ** 28 // (batch * kv_heads * head_dim)  # tokens a sequence may hold
        return {**shape, "batch": batch, "q": 1, "len": _spread(rng, 16, min(131072, room))}
    q = _spread(rng, 2, min(4096, 2 ** 24 // (heads * head_dim)))
    batch = _spread(rng, 1, max(1, min(16, 2 ** 25 // (heads * head_dim * q))))
    room = min(2 ** 28 // (batch * kv_heads * head_dim), 2 ** 37 // (batch * heads * q * head_dim))
    return {**shape, "batch": batch, "q": q, "len": _spread(rng, q, max(q, min(16384, room)))}


def _spans(case):
    """(tokens a sequence holds in all, new tokens among them), one pair per
    sequence; fixed by the case alone, so that work() knows them."""
    rng = random.Random(case["batch"] * 1000003 + case["len"] * 1009 + case["q"])
    spans = []
    for b in range(case["batch"]):
        new = case["q"] if b == 0 else rng.randint(max(1, case["q"] // 8), case["q"])
        total = case["len"] if b == 0 else rng.randint(max(new, case["len"] // 4), max(new, case["len"]))
        spans.append((max(total, new), new))
    return spans


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    state = dict(case)
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        wide = 1 + 9 * (torch.rand(k, generator=gen, device="cuda") < 0.01)   # outlier channels
        state["x"] = normal(m, k).half()
        state["residual"] = (2 * normal(m, k) * wide).half()
        state["weight"] = (1 + 0.2 * normal(k)).half()
        return state
    if case["op"] == "swiglu":
        state["gate_up"] = (1.5 * normal(case["m"], 2 * case["k"])).half()
        return state

    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    spans = _spans(case)
    total = sum(new for _, new in spans)
    ends = [0]
    for _, new in spans:
        ends.append(ends[-1] + new)
    used = [-(-length // page) for length, _ in spans]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    place = torch.zeros(case["batch"], max(used), dtype=torch.int64)
    done = 0
    for b, n in enumerate(used):
        place[b, :n] = torch.arange(done, done + n)
        done += n
    state["block_table"] = order[place.cuda()]
    state["seq_lens"] = torch.tensor([length for length, _ in spans], dtype=torch.int32).cuda()
    state["cu_q"] = torch.tensor(ends, dtype=torch.int32).cuda()
    state["max_len"] = max(length for length, _ in spans)
    state["kv_cache"] = torch.empty(pages, 2, kv_heads, page, dim, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 27) // (2 * kv_heads * page * dim))
    for at in range(0, pages, step):
        part = state["kv_cache"][at:at + step]
        part.copy_((34 * normal(*part.shape)).round_().clamp_(-127, 127))
    size = 0.6 + 0.8 * torch.rand(pages, 2, kv_heads, generator=gen, device="cuda")
    state["kv_scale"] = (size / 34).half()
    if case["op"] == "append":
        channel = 1 + 3 * (torch.rand(dim, generator=gen, device="cuda") < 0.05)   # outlier channels
        qkv = normal(total, heads + 2 * kv_heads, dim)
        qkv[:, heads:heads + kv_heads] *= channel
        state["qkv"] = qkv.half().view(total, -1)
        half = case["rotary"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(state["max_len"], dtype=torch.float64, device="cuda")[:, None] * freq
        state["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        return state
    state["queries"] = (2 * normal(total, heads, dim)).half()
    state["scale"] = dim ** -0.5
    return state


# --------------------------------------------------------------------- run
def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state)


def _run_own(s):
    import w4a8_gemm_amd as w4
    if s["op"] == "norm":
        h, a8, s_a = w4.rms_norm_quant(s["x"], s["weight"], EPS, residual=s["residual"])
        return {"h": h, "a": a8 * s_a[:, None]}
    if s["op"] == "swiglu":
        a8, s_a = w4.silu_mul_quant(s["gate_up"])
        return {"a": a8 * s_a[:, None]}
    cu_q = s["cu_q"] if s["q"] > 1 else None
    if s["op"] == "append":
        heads, kv_heads, dim = s["heads"], s["kv_heads"], s["head_dim"]
        q, k, v = s["qkv"].view(-1, heads + 2 * kv_heads, dim).split([heads, kv_heads, kv_heads], dim=1)
        q = w4.rope_append(q, k, v, s["cos_sin"], s["kv_cache"], s["kv_scale"], s["block_table"],
                           s["seq_lens"], cu_q=cu_q, interleaved=s["interleaved"])
        return {"q": q, "kv": s["kv_cache"] * s["kv_scale"][..., None, None]}
    return {"o": w4.paged_attention(s["queries"], s["kv_cache"], s["kv_scale"], s["block_table"],
                                    s["seq_lens"], cu_q=cu_q, max_q=s["q"], max_len=s["max_len"],
                                    scale=s["scale"], window=s["window"])}


def _int8_rows(y):
    """Values that per-token int8 codes and fp16 scales of the rows stand for."""
    scale = (y.abs().amax(dim=1, keepdim=True) / 127).half().float()
    recip = torch.where(scale > 0, 1 / scale, 0.0)
    return ((y * recip).round().clamp(-127, 127) * scale).half()


def _plain_norm(s):
    h = (s["x"].float() + s["residual"].float()).half()
    x = h.float()
    rstd = torch.rsqrt(x.square().mean(dim=1, keepdim=True) + EPS)
    return {"h": h, "a": _int8_rows(x * rstd * s["weight"].float())}


def _plain_swiglu(s):
    gate, up = s["gate_up"].float().split(s["k"], dim=1)
    return {"a": _int8_rows(gate / (1 + torch.exp(-gate)) * up)}


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dim] with its first 2 * cos.shape[-1] values rotated."""
    half = cos.shape[-1]
    part = x[..., :2 * half]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = part[..., :half], part[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., 2 * half:]], dim=-1)


def _plain_append(s):
    heads, kv_heads, dim, page = s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    cache, scales, cu, lens = s["kv_cache"], s["kv_scale"], s["cu_q"], s["seq_lens"]
    qkv = s["qkv"].view(-1, heads + 2 * kv_heads, dim).float()
    total, pages = qkv.shape[0], cache.shape[0]
    token = torch.arange(total, device=cu.device, dtype=torch.int32)
    seq = torch.bucketize(token, cu[1:], right=True)
    pos = (lens[seq] - cu[seq + 1] + token).long()
    where, slot = s["block_table"][seq, pos // page].long(), pos % page

    half = s["rotary"] // 2
    cos, sin = s["cos_sin"][pos][:, None, :half], s["cos_sin"][pos][:, None, half:]
    turned = _rotate(qkv[:, :heads + kv_heads], cos, sin, s["interleaved"])
    kv = torch.stack([turned[:, heads:], qkv[:, heads + kv_heads:]], dim=1)   # [token, 2, head, dim]

    # each written page's scale: the larger of its old one (if it held tokens
    # before the first new one) and the new tokens' own
    largest = torch.zeros(pages, 2, kv_heads, device=cu.device)
    largest.index_reduce_(0, where, kv.abs().amax(dim=-1), "amax")
    first = torch.full((pages,), page, device=cu.device).index_reduce_(0, where, slot, "amin")
    written, kept = (first < page)[:, None, None], ((first > 0) & (first < page))[:, None, None]
    before = torch.where(kept, scales.float(), 0.0)
    after = torch.where(written, torch.maximum(before, (largest / 127).half().float()), scales.float())
    # codes that were there, in the new scale
    ratio = torch.where(kept & (after > 0), before / after, 1.0)[..., None, None]
    held = torch.arange(page, device=cu.device)[:, None] < first[:, None, None, None, None]
    codes = torch.where(held & kept[..., None, None], (cache * ratio).round(), cache.float())
    # and the new ones
    recip = torch.where(after > 0, 1 / after, 0.0)
    codes[where, :, :, slot] = (kv * recip[where][..., None]).round().clamp(-127, 127)
    cache.copy_(codes)
    scales.copy_(after)
    return {"q": turned[:, :heads].half(), "kv": (codes * after[..., None, None]).half()}


def _plain_attention(s):
    heads, kv_heads, dim, page = s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    cu, lens, table = s["cu_q"].long(), s["seq_lens"].long(), s["block_table"].long()
    batch, most, length, group = s["batch"], s["q"], table.shape[1] * page, heads // kv_heads
    q, total = s["queries"], s["queries"].shape[0]

    def gathered(which):   # [batch, kv_heads, length, dim]
        values = s["kv_cache"][:, which][table] * s["kv_scale"][:, which][table].float()[..., None, None]
        return values.transpose(1, 2).reshape(batch, kv_heads, length, dim)

    # queries padded to [batch, kv_heads, group * most, dim]
    new = cu[1:] - cu[:-1]
    step = torch.arange(most, device=cu.device)
    rows = (cu[:-1, None] + step).clamp(max=total - 1)
    padded = q[rows].float().view(batch, most, kv_heads, group, dim).permute(0, 2, 3, 1, 4)
    padded = padded.reshape(batch, kv_heads, group * most, dim)

    scores = torch.matmul(padded, gathered(0).transpose(2, 3).contiguous()).mul_(s["scale"])
    pos = (lens - new)[:, None] + step                       # [batch, most]
    key = torch.arange(length, device=cu.device)
    seen = (key <= pos[..., None]) & (key < lens[:, None, None])
    if s["window"]:
        seen &= key > pos[..., None] - s["window"]
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


_PLAIN = {"norm": _plain_norm, "swiglu": _plain_swiglu, "append": _plain_append,
          "attention": _plain_attention}


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "norm":      # x, residual in; h, codes, scales out
        m, k = case["m"], case["k"]
        return {"bytes": m * k * (2 + 2 + 2 + 1) + 2 * k + 2 * m, "flops": 8 * m * k}
    if case["op"] == "swiglu":
        m, k = case["m"], case["k"]
        return {"bytes": m * k * (2 + 2 + 1) + 2 * m, "flops": 8 * m * k}
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    spans = _spans(case)
    total = sum(new for _, new in spans)
    if case["op"] == "append":
        written = sum(-(-length // page) - (length - new) // page for length, new in spans)
        moved = total * dim * (heads * 4 + kv_heads * 2 * 3)
        return {"bytes": moved + total * case["rotary"] * 4 + written * kv_heads * 2 * 4,
                "flops": total * dim * (3 * heads + 2 * kv_heads * 4)}
    window = case["window"]
    read = pairs = 0
    for length, new in spans:
        first = length - new                     # position of the first query
        read += length - (max(0, first + 1 - window) if window else 0)
        reach = [0, 0]                           # keys seen by all queries at positions < p
        for i, p in enumerate((first, length)):
            full = min(p, window) if window else p
            reach[i] = full * (full + 1) // 2 + (p - full) * window
        pairs += reach[1] - reach[0]
    return {"bytes": read * kv_heads * 2 * (dim + 2 / page) + total * heads * dim * 4,
            "flops": 4 * heads * dim * pairs}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, row by row and
    sequence by sequence."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "swiglu": _exact_swiglu, "append": _exact_append,
            "attention": _exact_attention}[case["op"]](s)


def _exact_codes(values, scale):
    """round(values / scale) within +-127, 0 under a zero scale (64 bits)."""
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = torch.clamp(torch.round(values / safe), -127, 127)
    return torch.where(scale > 0, codes, torch.zeros_like(codes))


def _exact_scale(largest):
    return (largest / 127).to(torch.float16).double()


def _exact_norm(s):
    h = (s["x"].double() + s["residual"].double()).to(torch.float16)
    y = torch.empty(h.shape, dtype=torch.float64, device=h.device)
    for at in range(0, h.shape[0], 1024):
        row = h[at:at + 1024].double()
        length = torch.sqrt((row * row).sum(1) / row.shape[1] + EPS)
        normed = row / length.unsqueeze(1) * s["weight"].double()
        scale = _exact_scale(normed.abs().max(1).values).unsqueeze(1)
        y[at:at + 1024] = _exact_codes(normed, scale) * scale
    return {"h": h.double(), "a": y}


def _exact_swiglu(s):
    gate, up = s["gate_up"][:, :s["k"]].double(), s["gate_up"][:, s["k"]:].double()
    y = gate * torch.sigmoid(gate) * up
    scale = _exact_scale(y.abs().max(1).values).unsqueeze(1)
    return {"a": _exact_codes(y, scale) * scale}


def _exact_append(s):
    heads, kv_heads, dim, page = s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    codes, scales = s["kv_cache"].double(), s["kv_scale"].double()
    qkv = s["qkv"].double().view(-1, heads + 2 * kv_heads, dim)
    half = s["rotary"] // 2
    q_out = []
    ends, lens, table = s["cu_q"].tolist(), s["seq_lens"].tolist(), s["block_table"].tolist()
    for b in range(s["batch"]):
        part = qkv[ends[b]:ends[b + 1]].clone()
        n, start = part.shape[0], lens[b] - part.shape[0]
        # rotation as a product of complex numbers
        turn = torch.complex(s["cos_sin"][start:start + n, :half].double(),
                             s["cos_sin"][start:start + n, half:].double()).unsqueeze(1)
        first = torch.arange(half, device=part.device) * (2 if s["interleaved"] else 1)
        second = first + (1 if s["interleaved"] else half)
        both = part[:, :heads + kv_heads]
        z = torch.complex(both[..., first], both[..., second]) * turn
        both[..., first], both[..., second] = z.real, z.imag
        q_out.append(part[:, :heads])
        kv = part[:, heads:].reshape(n, 2, kv_heads, dim)
        for index in range(start // page, (lens[b] - 1) // page + 1):
            at, lo = table[b][index], max(start, index * page)
            hi = min(lens[b], index * page + page)
            fresh = kv[lo - start:hi - start]                        # [tokens, 2, head, dim]
            scale = _exact_scale(fresh.abs().amax((0, 3)))           # [2, head]
            there = lo - index * page
            if there:
                old = scales[at].clone()
                scale = torch.maximum(scale, old)
                held = codes[at, :, :, :there] * old[:, :, None, None]
                codes[at, :, :, :there] = _exact_codes(held, scale[:, :, None, None])
            scales[at] = scale
            fresh = fresh.permute(1, 2, 0, 3)
            codes[at, :, :, there:hi - index * page] = _exact_codes(fresh, scale[:, :, None, None])
    return {"q": torch.cat(q_out), "kv": codes * scales[..., None, None]}


def _exact_attention(s):
    heads, kv_heads, dim, page = s["heads"], s["kv_heads"], s["head_dim"], s["page"]
    if work({k: s[k] for k in s if not torch.is_tensor(s[k])})["flops"] > 2e12:
        return None
    out = torch.zeros(s["queries"].shape, dtype=torch.float64, device=s["queries"].device)
    ends, lens = s["cu_q"].tolist(), s["seq_lens"].tolist()
    group = heads // kv_heads
    for b in range(s["batch"]):
        lo, hi, length = ends[b], ends[b + 1], lens[b]
        at = s["block_table"][b, :-(-length // page)].long()
        for head in range(kv_heads):
            code = s["kv_cache"][at, :, head].double() * s["kv_scale"][at, :, head].double()[..., None, None]
            key = code[:, 0].reshape(-1, dim)[:length]
            value = code[:, 1].reshape(-1, dim)[:length]
            for g in range(head * group, (head + 1) * group):
                score = s["queries"][lo:hi, g].double() @ key.t().contiguous() * s["scale"]
                back = torch.arange(length - hi + lo, length, device=key.device)[:, None] \
                    - torch.arange(length, device=key.device)
                hidden = back < 0
                if s["window"]:
                    hidden |= back >= s["window"]
                score[hidden] = float("-inf")
                out[lo:hi, g] = torch.softmax(score, dim=1) @ value
    return {"o": out}
