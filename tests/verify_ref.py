"""Plain numpy implementations, in 64 bits, of the operators that verify and end a
decoding step: the yardstick of their GPU tests."""
import numpy as np

from decoder_ref import half_ulp16


# -------------------------------------------------------------------- trees
def random_parents(n, rng, roots=False):
    """A random tree of n nodes, parents before children; with `roots` some
    nodes have none."""
    return [-1 if i == 0 or (roots and rng.random() < 0.1) else int(i * rng.random() ** 1.5) for i in range(n)]


def ancestors(parents):
    """[n, n] bool: node i sees node j."""
    n = len(parents)
    see = np.zeros((n, n), bool)
    for i in range(n):
        if 0 <= parents[i] < i:
            see[i] = see[parents[i]]
        see[i, i] = True
    return see


def pack_mask(see, words):
    """[n, m] bool as int32 words; columns beyond 32 * words are dropped."""
    wide = np.zeros((see.shape[0], 32 * words), np.uint64)
    m = min(see.shape[1], 32 * words)
    wide[:, :m] = see[:, :m]
    return (wide.reshape(see.shape[0], words, 32) << np.arange(32, dtype=np.uint64)).sum(axis=2).astype(np.uint32).view(np.int32)


def seen_positions(see_row, start, window):
    """Positions that a row sees: the cached ones and the nodes of its mask row,
    the last `window` of them where there is one."""
    keys = np.concatenate([np.arange(max(start, 0)), start + np.flatnonzero(see_row)])
    keys = keys[keys >= 0]
    return keys[-window:] if window else keys


def tree_attention(q, cache, scale_kv, table, lens, cu, see, scale, window=0):
    """(o, bound) float64: see[b] is the [n, n] mask of sequence b.  The bound is
    decoder_ref.attention()'s: half an fp16 ulp of the result, 2^-11 of each
    softmax weight, and scores off by dim + 8 roundings of fp32."""
    tokens, heads, dim = q.shape
    pages, _, kv_heads, page, _ = cache.shape
    group = heads // kv_heads
    out = np.zeros((tokens, heads, dim))
    bound = np.full((tokens, heads, dim), half_ulp16(0))
    for b in range(len(lens)):
        n, length = cu[b + 1] - cu[b], int(lens[b])
        ids = np.array([int(table[b, i]) for i in range(-(-length // page))], dtype=np.int64)
        there = np.repeat((ids >= 0) & (ids < pages), page)[:length]
        ids = np.where((ids >= 0) & (ids < pages), ids, 0)
        for h in range(kv_heads):
            if not len(ids):
                continue
            code = cache[ids][:, :, h].astype(np.float64) * scale_kv[ids][:, :, h].astype(np.float64)[..., None, None]
            k, v = code[:, 0].reshape(-1, dim)[:length], code[:, 1].reshape(-1, dim)[:length]
            for i in range(n):
                keys = seen_positions(see[b][i], length - n, window)
                keys = keys[there[keys]]
                if not len(keys):
                    continue
                rows = q[cu[b] + i, h * group:(h + 1) * group].astype(np.float64)
                x = rows @ k[keys].T * scale
                p = np.exp(x - x.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                o = p @ v[keys]
                d = (np.abs(rows) @ np.abs(k[keys]).T).max(axis=1, keepdims=True) * abs(scale) * (dim + 8) * 2.0 ** -24
                at = cu[b] + i, slice(h * group, (h + 1) * group)
                out[at] = o
                bound[at] = half_ulp16(np.abs(o)) * 1.001 + (p @ np.abs(v[keys])) * (2.0 ** -11 + np.expm1(2 * d) + 2.0 ** -19)
    return out, bound


def accept(drafted, parents, sampled, n, most):
    """(path, next token) of one tree of n nodes."""
    if n == 0:
        return [], -1
    path = [0]
    while len(path) < most and sampled[path[-1]] >= 0:
        fits = [c for c in range(path[-1] + 1, n) if parents[c] == path[-1] and drafted[c] == sampled[path[-1]]]
        if not fits:
            break
        path.append(fits[0])
    return path, int(sampled[path[-1]])


def keep(cache, scale, table, lens, cu, paths):
    """(codes before rounding float64, scale float16, moved [pages, page] bool) of
    a cache after confirmed nodes have moved; slots that are not written or
    rescaled keep their codes."""
    pages, _, kv_heads, page, dim = cache.shape
    codes, new = cache.astype(np.float64), scale.copy()
    touched = np.zeros((pages, page), bool)
    at_page = lambda b, pos: int(table[b, pos // page]) if pos // page < table.shape[1] and 0 <= table[b, pos // page] < pages else -1
    for b, path in enumerate(paths):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        if start < 0:
            continue
        for index in range(start // page, (start + len(path) - 1) // page + 1 if path else 0):
            to = at_page(b, index * page)
            inside = [i for i in range(len(path)) if (start + i) // page == index and i <= path[i] < n
                      and at_page(b, start + path[i]) >= 0]
            if to < 0 or not inside:
                continue
            held = max(0, start - index * page)
            sources = [at_page(b, start + path[i]) for i in inside] + ([to] if held else [])
            s = np.max([scale[p] for p in sources], axis=0)
            new[to] = s
            s = s.astype(np.float64)
            ratio = lambda p: np.where(scale[p] == new[to], 1.0, scale[p].astype(np.float64) / np.where(s > 0, s, 1.0))[..., None]
            for slot in range(held):
                codes[to, :, :, slot] = cache[to, :, :, slot] * ratio(to)
                touched[to, slot] = True
            for i in inside:
                p = at_page(b, start + path[i])
                codes[to, :, :, (start + i) % page] = cache[p, :, :, (start + path[i]) % page] * ratio(p)
                touched[to, (start + i) % page] = True
    return codes, new, touched


# ----------------------------------------------------------------- sampling
def sample(x, u, temperature, top_k, top_p, min_p):
    """(token, share) of one row of float64 logits."""
    if np.isnan(x).any() or np.isposinf(x).any():
        return -1, np.nan
    if np.isneginf(x).all():
        return -1, 0.0
    if temperature == 0:
        return int(np.argmax(x)), 1.0
    order = np.argsort(-x, kind="stable")
    if 0 < top_k < len(x):
        order = order[:top_k]
    with np.errstate(over="ignore", under="ignore"):
        w = np.exp((x[order] - x.max()) / temperature)
    n = len(order)
    if top_p < 1:
        upto = np.cumsum(w)
        n = min(n, int(np.searchsorted(upto, max(top_p, 0.0) * upto[-1])) + 1)
    n = min(n, int((w >= min(max(min_p, 0.0), 1.0)).sum()))
    chosen = np.argsort(order[:n], kind="stable")
    ids, w = order[:n][chosen], w[:n][chosen]
    upto = np.cumsum(w)
    u = 0.0 if not u >= 0 else min(u, 1 - 2.0 ** -24)
    at = int(np.searchsorted(upto, u * upto[-1], side="right"))
    return int(ids[at]), w[at] / upto[-1]


# -------------------------------------------------------------------- pages
def valid(p, pages):
    return p if 0 <= p < pages else -1


def fork(table, lens, refs, parent, page):
    table, refs = table.tolist(), refs.tolist()
    pages, width = len(refs), len(table[0]) if table else 0
    rows, ends = [], []
    for i, j in enumerate(parent):
        if not 0 <= j < len(table):
            rows.append([-1] * width)
            ends.append(0)
            continue
        used = -(-min(max(lens[j], 0), width * page) // page)
        rows.append([valid(p, pages) if i == j or c < used else -1 for c, p in enumerate(table[j])])
        ends.append(int(lens[j]))
    for lines, sign in ((table, -1), (rows, 1)):
        for line in lines:
            for p in line:
                if valid(p, pages) >= 0:
                    refs[p] += sign
    return np.array(rows, np.int32).reshape(len(parent), width), np.array(ends, np.int32), np.array(refs, np.int32)


def alloc(table, lens, refs, tokens, page):
    """table, lens, refs, pairs, missing."""
    pages, width = len(refs), table.shape[1]
    fixed, refs = refs.tolist(), refs.tolist()
    free = [p for p, n in enumerate(fixed) if n <= 0]
    before = [[valid(p, pages) for p in line] for line in table.tolist()]
    rows = [list(line) for line in before]
    lens = [min(max(int(n), 0), width * page) for n in lens]
    writes = [lens[b] % page != 0 and tokens[b] > 0 for b in range(len(rows))]
    pairs, missing = [], 0
    for b, line in enumerate(rows):
        end = -(-(lens[b] + max(tokens[b], 0)) // page) if tokens[b] > 0 else 0
        for c in range(lens[b] // page, end):
            if c >= width:
                missing += 1
                continue
            p = before[b][c]
            if p >= 0:
                if c > lens[b] // page or not writes[b] or fixed[p] < 2:
                    continue
                holders = [r for r in range(len(rows)) if writes[r] and lens[r] // page < width and before[r][lens[r] // page] == p]
                if len(holders) >= fixed[p] and holders[-1] == b:
                    continue
                refs[p] -= 1
            line[c] = free.pop(0) if free else -1
            missing += line[c] < 0
            if line[c] >= 0:
                refs[line[c]] = 1
                if p >= 0:
                    pairs.append((p, line[c]))
    ends = [n + max(t, 0) for n, t in zip(lens, tokens)]
    return (np.array(rows, np.int32).reshape(len(rows), width), np.array(ends, np.int32), np.array(refs, np.int32),
            pairs, missing)


def compact(table, refs):
    """table, refs, place, pairs."""
    pages, refs = len(refs), refs.tolist()
    live = sum(n > 0 for n in refs)
    pairs = list(zip([p for p in range(live, pages) if refs[p] > 0], [p for p in range(live) if refs[p] <= 0]))
    place = list(range(pages))
    for source, target in pairs:
        place[source] = target
        refs[target], refs[source] = refs[source], 0
    rows = [[place[p] if valid(p, pages) >= 0 else -1 for p in line] for line in table.tolist()]
    return (np.array(rows, np.int32).reshape(table.shape), np.maximum(np.array(refs, np.int32), 0),
            np.array(place, np.int32), pairs)
