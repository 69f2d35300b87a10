"""Trees of drafted tokens on the GPU against 64-bit numpy: masks and positions,
attention, the confirmed path, and its keys and values moved together."""
import numpy as np
import pytest

import decoder_ref as dref
import verify_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import device, log
from test_gpu_kv_cache import Batch, append, check_append

pytestmark = pytest.mark.gpu


def put(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def trees(batch, roots=False):
    """Random trees for the new tokens of a Batch: (parents [tokens], masks)."""
    each = [ref.random_parents(n, batch.rng, roots) for _, n in batch.spans]
    return np.array([p for e in each for p in e], np.int32), [ref.ancestors(e) for e in each]


def mask_of(see, words):
    rows = [ref.pack_mask(s, words) for s in see if len(s)]
    return np.concatenate(rows) if rows else np.zeros((0, words), np.int32)


def attend(batch, q, mask, dev, window=0, state=None, **kw):
    import torch
    st = state or batch.device(dev)
    q = q if torch.is_tensor(q) else put(q, dev)
    o = w4.tree_attention(q, st["cache"], st["scale"], st["block_table"], st["seq_lens"],
                          mask if torch.is_tensor(mask) else put(mask, dev), cu_q=st["cu_q"], window=window, **kw)
    torch.cuda.synchronize()
    return o.cpu().numpy()


def check(batch, q, see, o, window=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, bound = ref.tree_attention(q, batch.cache, batch.scale, batch.table, batch.lens, batch.cu, see, scale, window)
    err = np.abs(o.astype(np.float64) - want)
    assert (err <= bound).all(), (np.unravel_index((err - bound).argmax(), err.shape), (err / bound).max())


SPANS = [(70, 70), (5, 1), (200, 33), (64, 0), (0, 0), (17, 17), (129, 2), (300, 64), (1, 1), (257, 130), (95, 32)]


def test_mask_and_positions():
    dev = device()
    log("tree mask")
    batch = Batch(SPANS, 16, 1, 16, 1)
    parents, see = trees(batch, roots=True)
    parents[0] = 5                                   # a parent that comes later is none
    parents[75] = 1 << 30
    each = [parents[lo:hi] for lo, hi in zip(batch.cu, batch.cu[1:])]
    see = [ref.ancestors(list(e)) for e in each]
    lens, cu = put(batch.lens, dev), put(batch.cu, dev)
    for words, kw in ((11, {}), (5, dict(max_q=130)), (1, dict(max_q=20))):
        mask, positions = w4.tree_mask(put(parents, dev), lens, cu_q=cu, **kw)
        assert mask.shape == (batch.tokens, words)
        assert (mask.cpu().numpy() == mask_of(see, words)).all()
        depth = np.concatenate([s.sum(axis=1) - 1 for s in see if len(s)])
        start = np.concatenate([np.full(n, length - n) for length, n in batch.spans])
        assert (positions.cpu().numpy() == start + depth).all()
    one, positions = w4.tree_mask(put(np.full(11, -1, np.int32), dev), lens)          # one node each
    assert (one.cpu().numpy() == 1).all() and (positions.cpu().numpy() == batch.lens - 1).all()


@pytest.mark.parametrize("window", [0, 1, 7, 40, 1000])
@pytest.mark.parametrize("page,heads,kv_heads,dim", [(16, 8, 2, 128), (64, 4, 4, 64), (32, 6, 2, 80), (128, 5, 1, 256),
                                                     (16, 17, 1, 96), (64, 32, 1, 128), (16, 3, 1, 16), (32, 2, 2, 192)])
def test_attention(page, heads, kv_heads, dim, window):
    dev = device()
    log(f"tree attention page={page} heads={heads}/{kv_heads} dim={dim} window={window}")
    batch = Batch(SPANS, page, kv_heads, dim, 2)
    parents, see = trees(batch, roots=True)
    q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
    mask, _ = w4.tree_mask(put(parents, dev), put(batch.lens, dev), cu_q=put(batch.cu, dev), max_q=130)
    check(batch, q, see, attend(batch, q, mask, dev, window), window)


@pytest.mark.parametrize("most", [None, 1, 9, 130])
@pytest.mark.parametrize("window", [0, 3, 60])
def test_any_mask(window, most):
    """Masks that are no trees: rows without their own bit, empty rows (0 where
    there is no cached token either), bits beyond the sequence's nodes; bounds
    that are too small or too large."""
    dev = device()
    log(f"tree attention any mask window={window} max_q={most}")
    batch = Batch(SPANS, 16, 2, 128, 3)
    see = [batch.rng.random((n, n)) < batch.rng.choice([0.05, 0.5, 0.95], (n, 1)) for _, n in batch.spans]
    for s in see:
        if len(s):
            s[batch.rng.integers(len(s))] = False
    see[0][:] &= np.arange(70)[:, None] % 3 > 0        # no cached tokens: a third of the rows sees nothing
    wide = [np.concatenate([s, np.ones((len(s), 160 - len(s)), bool)], axis=1) for s in see]
    q = (2 * batch.rng.standard_normal((batch.tokens, 6, 128))).astype(np.float16)
    o = attend(batch, q, mask_of(wide, 5), dev, window, max_q=most)
    check(batch, q, see, o, window)
    assert (o[:70][::3] == 0).all() and (o[1:70][::3] != 0).any()


def test_mask_words_that_do_not_reach_all_nodes():
    dev = device()
    log("tree attention few words")
    batch = Batch(SPANS, 32, 2, 64, 4)
    _, see = trees(batch)
    q = batch.rng.standard_normal((batch.tokens, 4, 64)).astype(np.float16)
    cut = [s & (np.arange(len(s)) < 64) for s in see]
    check(batch, q, cut, attend(batch, q, mask_of(see, 2), dev))


@pytest.mark.parametrize("heads,kv_heads,dim,nodes", [(4, 1, 128, 3), (2, 2, 64, 40), (6, 1, 256, 9), (8, 1, 128, 31)])
@pytest.mark.parametrize("length", [300, 2049, 9000])
def test_split_over_a_long_sequence(length, heads, kv_heads, dim, nodes):
    """Few rows over many keys: the splits' join, also where the host's bound
    is far off."""
    dev = device()
    for bound, window in ((None, 0), (64, 0), (length, 700), (20 * length, 0)):
        log(f"tree attention long={length} heads={heads}/{kv_heads} dim={dim} nodes={nodes} max_len={bound}")
        batch = Batch([(length, nodes), (3, 2), (7, 7), (0, 0)], 64, kv_heads, dim, 5, wide=40)
        _, see = trees(batch)
        q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
        check(batch, q, see, attend(batch, q, mask_of(see, 2), dev, window, max_len=bound, max_q=nodes), window)


def test_one_node_each_without_cu_q():
    dev = device()
    log("tree attention one node")
    for group in (1, 4, 20, 40):
        batch = Batch([(n, 1) for n in (1, 2, 17, 33, 100, 600)], 16, 2, 128, 6, cu=False)
        q = batch.rng.standard_normal((6, 2 * group, 128)).astype(np.float16)
        check(batch, q, [np.ones((1, 1), bool)] * 6, attend(batch, q, np.ones((6, 1), np.int32), dev))
    # the node itself not seen: the first sequence sees nothing
    o = attend(batch, q, np.zeros((6, 1), np.int32), dev)
    check(batch, q, [np.zeros((1, 1), bool)] * 6, o)
    assert (o[0] == 0).all()


@pytest.mark.parametrize("count,nodes,dim", [(65, 3, 64), (130, 20, 16), (300, 1, 32), (5000, 1, 16), (4500, 2, 16)])
def test_many_sequences(count, nodes, dim):
    """More sequences than lanes, some of them long (so that their tiles are split
    where that is done at all), some without nodes."""
    dev = device()
    log(f"tree attention {count} sequences of up to {nodes}")
    rng = np.random.default_rng(21)
    spans = [(int(n) + int(rng.integers(0, 40)), int(n)) for n in rng.integers(0, nodes + 1, count)]
    spans[count // 2] = (3000, nodes)
    spans[-1] = (2000, nodes)
    batch = Batch(spans, 64, 1, dim, 22)
    _, see = trees(batch)
    q = batch.rng.standard_normal((batch.tokens, 2, dim)).astype(np.float16)
    for most in (None, 100):
        check(batch, q, see, attend(batch, q, mask_of(see, 1), dev, max_q=nodes, max_len=most))


def test_tables_that_are_improper():
    """cu_q that does not ascend or ends beyond the rows, lengths and pages out of
    range: nothing outside the buffers is touched (results mean nothing), and what
    the other sequences get is untouched memory or finite."""
    import torch
    dev = device()
    log("tree attention improper tables")
    batch = Batch([(100, 20), (40, 10), (64, 10)], 16, 2, 64, 23)
    q = batch.rng.standard_normal((40, 4, 64)).astype(np.float16)
    mask = np.full((40, 1), -1, np.int32)
    for cu in ([0, 40, 10, 40], [5, 2, 1, 0], [0, 100, 200, 300], [-7, 40, 40, 90], [2 ** 31 - 1] * 4, [-2 ** 31] * 4):
        for lens in ([100, 40, 64], [-5, 2 ** 31 - 1, 10], [0, 0, 0]):
            st = batch.device(dev)
            st["cu_q"], st["seq_lens"] = put(np.array(cu, np.int32), dev), put(np.array(lens, np.int32), dev)
            guard = torch.full((42, 4, 64), 7.0, dtype=torch.float16, device=dev)
            attend(batch, q, mask, dev, state=st, out=guard[1:41])
            w4.tree_mask(put(np.zeros(40, np.int32), dev), st["seq_lens"], cu_q=st["cu_q"])
            path, count, _, _ = w4.tree_accept(put(np.zeros(40, np.int32), dev), put(np.zeros(40, np.int32), dev),
                                               put(np.zeros(40, np.int32), dev), st["seq_lens"], cu_q=st["cu_q"])
            w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], path, count, cu_q=st["cu_q"])
            torch.cuda.synchronize()
            assert (guard[0] == 7).all() and (guard[41] == 7).all()


def test_values_that_are_not_ordinary():
    """NaN in a query stays in its rows; a row that sees nothing is 0 all the
    same; scales of pages that are not seen do not reach a row; absent pages are
    not seen; large scores, scale 0."""
    dev = device()
    log("tree attention not ordinary")
    batch = Batch([(100, 20), (40, 40), (64, 10)], 16, 2, 128, 7)
    _, see = trees(batch)
    see[1][3] = False
    q = (2 * batch.rng.standard_normal((batch.tokens, 4, 128))).astype(np.float16)
    batch.table[0, 2] = -1
    batch.table[2, 1] = batch.pages + 3
    batch.scale[batch.table[2, 0], 1, 0] = 0           # values of that page are 0
    q[5, 1, 7], q[21, 2, 0], q[23, 0, 5] = np.nan, np.inf, np.nan
    o = attend(batch, q, mask_of(see, 2), dev)
    assert np.isnan(o[5, 1]).all() and np.isnan(o[21, 2]).all() and (o[23, 0] == 0).all()
    clean = q.copy()
    clean[5, 1], clean[21, 2], clean[23, 0] = 0, 0, 0
    o[5, 1], o[21, 2] = 0, 0
    want, bound = ref.tree_attention(clean, batch.cache, batch.scale, batch.table, batch.lens, batch.cu, see, 128 ** -0.5)
    err = np.abs(o.astype(np.float64) - want)
    err[5, 1], err[21, 2] = 0, 0
    assert (err <= bound).all()
    # a NaN scale where only some rows look: the last nodes' page of sequence 1
    batch = Batch([(40, 40)], 16, 1, 64, 8)
    see = [np.tril(np.ones((40, 40), bool))]
    q = batch.rng.standard_normal((40, 1, 64)).astype(np.float16)
    batch.scale[batch.table[0, 2]] = np.nan
    o = attend(batch, q, mask_of(see, 2), dev)
    assert np.isfinite(o[:32]).all() and np.isnan(o[32:]).all()
    # scores far beyond 2^27, negative score scale: where the largest of a row leads by
    # more than scores may be off (dim + 8 roundings each) and 40 besides, the row
    # is that key's value, within two roundings to fp16 (weight and result)
    batch = Batch([(90, 30)], 16, 1, 64, 9)
    _, see = trees(batch)
    q = (200 * batch.rng.standard_normal((30, 2, 64))).astype(np.float16)
    code = batch.cache[batch.table[0, :6]].astype(np.float64) * batch.scale[batch.table[0, :6]].astype(np.float64)[..., None, None]
    k, v = (code[:, i, 0].reshape(-1, 64) for i in (0, 1))
    for scale in (1e8, -3.0):
        o = attend(batch, q, mask_of(see, 1), dev, scale=scale).astype(np.float64)
        assert np.isfinite(o).all()
        led = 0
        for i in range(30):
            keys = ref.seen_positions(see[0][i], 60, 0)
            for h in range(2):
                x = q[i, h].astype(np.float64) @ k[keys].T * scale
                off = 2 * (np.abs(q[i, h].astype(np.float64)) @ np.abs(k[keys]).T).max() * abs(scale) * 72 * 2.0 ** -24
                best, second = np.sort(x)[[-1, -2]]
                if best - second > off + 40:
                    led += 1
                    want = v[keys[x.argmax()]]
                    assert (np.abs(o[i, h] - want) <= 2.0 ** -10 * np.abs(want) + 2.0 ** -24).all()
        assert led > 20


def test_strides_rows_behind_and_own_buffers():
    """Rows, masks and outputs with strides of their own; rows behind the last
    sequence are not written, with and without a split."""
    import torch
    dev = device()
    for length in (60, 5000):
        log(f"tree attention strides len={length}")
        batch = Batch([(length, 9), (30, 12)], 16, 2, 64, 10)
        _, see = trees(batch)
        q = batch.rng.standard_normal((21, 4, 64)).astype(np.float16)
        wide_q = torch.zeros((26, 8, 64), dtype=torch.float16, device=dev)
        wide_q[:21, 2:6] = put(q, dev)
        out = torch.full((26, 8, 64), 7.0, dtype=torch.float16, device=dev)
        mask = torch.full((26, 5), -1, dtype=torch.int32, device=dev)
        mask[:21, 1:2] = put(mask_of(see, 1), dev)
        st = batch.device(dev)
        o = w4.tree_attention(wide_q[:, 2:6], st["cache"], st["scale"], st["block_table"], st["seq_lens"], mask[:, 1:2],
                              cu_q=st["cu_q"], max_q=12, out=out[:, 2:6])
        torch.cuda.synchronize()
        check(batch, q, see, o[:21].cpu().numpy())
        assert (out[:, :2] == 7).all() and (out[:, 6:] == 7).all() and (out[21:] == 7).all()


def test_offsets_beyond_32_bits():
    """A cache whose pages lie 1.5 GiB apart: attention, append and keep at
    offsets beyond 2^32."""
    import torch
    dev = device()
    log("tree far pages")
    batch = Batch([(50, 10)], 16, 2, 64, 11, spare=0)
    far = torch.empty(4 * (3 << 29) + 4096, dtype=torch.int8, device=dev)
    cache = far.as_strided((4, 2, 2, 16, 64), (3 << 29, 2048, 1024, 64, 1))
    cache.copy_(put(batch.cache, dev))
    st = batch.device(dev)
    st["cache"] = cache
    parents, see = trees(batch)
    q = batch.rng.standard_normal((10, 4, 64)).astype(np.float16)
    check(batch, q, see, attend(batch, q, mask_of(see, 1), dev, state=st))
    paths = [[0, 3, 5, 9]]
    w4.kv_keep(cache, st["scale"], st["block_table"], st["seq_lens"], put(np.array(paths, np.int32), dev),
               put(np.array([4], np.int32), dev), cu_q=st["cu_q"])
    check_keep(batch, paths, cache.cpu().numpy(), st["scale"].cpu().numpy())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("spans", [[(70, 70), (5, 1), (200, 33), (0, 0)], [(9, 1), (64, 1), (17, 1)]])
def test_append_at_positions(spans, interleaved):
    """rope_append with given positions: as one with a table whose rows are
    those positions' in the places of the tokens."""
    import torch
    dev = device()
    log(f"append positions {spans}")
    cu = any(n != 1 for _, n in spans)
    batch = Batch(spans, 16, 2, 64, 12, cu=cu)
    table = w4.rope_table(300, 64, device=dev)
    positions = batch.rng.integers(-3, 310, batch.tokens).astype(np.int32)
    qkv = batch.rng.standard_normal((batch.tokens, 8, 64)).astype(np.float16)
    st = batch.device(dev)
    x = put(qkv, dev)
    q, k, v = x.split([4, 2, 2], dim=1)
    w4.rope_append(q, k, v, table, st["cache"], st["scale"], st["block_table"], st["seq_lens"], cu_q=st["cu_q"],
                   interleaved=interleaved, out=q, positions=put(positions, dev))
    torch.cuda.synchronize()
    # sequence by sequence with a table whose row at a token's place is its position's
    lo = 0
    for b, (length, n) in enumerate(spans):
        if n == 0:
            continue
        rows = np.zeros((length, 64), np.float32)
        rows[length - n:] = table.cpu().numpy()[np.clip(positions[lo:lo + n], 0, 299)]
        alone = Batch(spans, 16, 2, 64, 12, cu=cu)
        ast = alone.device(dev)
        got = put(qkv[lo:lo + n], dev)
        aq, ak, av = got.split([4, 2, 2], dim=1)
        at = torch.tensor([0, n], dtype=torch.int32, device=dev)
        w4.rope_append(aq, ak, av, torch.from_numpy(rows).to(dev), ast["cache"], ast["scale"],
                       ast["block_table"][b:b + 1], ast["seq_lens"][b:b + 1], cu_q=at, interleaved=interleaved, out=aq)
        torch.cuda.synchronize()
        assert torch.equal(aq, q[lo:lo + n])
        pages = ast["block_table"][b, :-(-length // 16)].long()
        assert torch.equal(ast["cache"][pages], st["cache"][pages])
        assert torch.equal(ast["scale"][pages], st["scale"][pages])
        lo += n


# ------------------------------------------------------------------- accept
def draft(spans, rng, vocab=3):
    """Trees over a small vocabulary, so that several children hold a token."""
    parents = [ref.random_parents(n, rng) for _, n in spans]
    drafted = [rng.integers(0, vocab, n) for _, n in spans]
    sampled = [rng.integers(0, vocab, n) for _, n in spans]
    return parents, drafted, sampled


@pytest.mark.parametrize("most", [None, 1, 3, 200])
def test_accept(most):
    dev = device()
    log(f"accept max_q={most}")
    rng = np.random.default_rng(13)
    spans = SPANS + [(400, 200), (90, 90), (1000, 1)] + [(50, int(n)) for n in rng.integers(0, 50, 40)]
    parents, drafted, sampled = draft(spans, rng)
    for chain in (0, len(SPANS)):                   # chains that are confirmed to the end
        n = spans[chain][1]
        parents[chain] = list(range(-1, n - 1))
        sampled[chain][:-1] = drafted[chain][1:]
    sampled[2][0] = -1                              # nothing drawn after the root,
    drafted[2][:] = -1                              # and tokens that equal it
    parents[6] = [7, 0]                             # a root with a parent
    flat = lambda x: put(np.concatenate([np.asarray(e) for e in x]).astype(np.int32), dev)
    cu = np.concatenate([[0], np.cumsum([n for _, n in spans])]).astype(np.int32)
    lens = np.array([length for length, _ in spans], np.int32)
    path, count, tokens, new = (t.cpu().numpy() for t in w4.tree_accept(
        flat(drafted), flat(parents), flat(sampled), put(lens, dev), cu_q=put(cu, dev), max_q=most))
    wide = max(1, min(cu[-1], most or cu[-1]))
    assert path.shape == (len(spans), wide)
    for b, (length, n) in enumerate(spans):
        want, token = ref.accept(drafted[b], parents[b], sampled[b], n, wide)
        assert path[b, :len(want)].tolist() == want and (path[b, len(want):] == -1).all()
        assert (count[b], tokens[b], new[b]) == (len(want), token, length - n + len(want))
    if most is None:
        assert count[0] == 70 and count[len(SPANS)] == 200
    # one node each: confirmed as it is
    one = put(np.arange(4, dtype=np.int32), dev)
    path, count, tokens, new = w4.tree_accept(one, one - 5, one + 7, one + 1)
    assert (path == 0).all() and (count == 1).all() and (tokens == one + 7).all() and (new == one + 1).all()


# --------------------------------------------------------------------- keep
def check_keep(batch, paths, cache, scale):
    codes, want_scale, touched = ref.keep(batch.cache, batch.scale, batch.table, batch.lens, batch.cu, paths)
    assert (scale.view(np.uint16) == want_scale.view(np.uint16)).all()
    # codes: the integer nearest to code * fp32(s / s'), two roundings of fp32
    near = np.abs(cache.astype(np.float64) - codes) <= 0.5 + 127 * 2.0 ** -22
    assert near.all()
    stay = ~touched
    assert (cache.transpose(0, 3, 1, 2, 4)[stay] == batch.cache.transpose(0, 3, 1, 2, 4)[stay]).all()


def random_paths(spans, rng, deep):
    return [[0] + sorted(rng.choice(np.arange(1, n), min(int(rng.integers(deep)), n - 1), replace=False).tolist())
            if n > 1 else [0] * n for _, n in spans]


@pytest.mark.parametrize("page,kv_heads,dim", [(16, 2, 128), (16, 3, 16), (64, 1, 256), (32, 4, 80), (1024, 2, 64)])
def test_keep(page, kv_heads, dim):
    import torch
    dev = device()
    for deep in (1, 6, 40, 200):
        log(f"keep page={page} heads={kv_heads} dim={dim} deep={deep}")
        batch = Batch(SPANS, page, kv_heads, dim, 14)
        paths = random_paths(batch.spans, batch.rng, deep)
        st = batch.device(dev)
        wide = np.full((len(paths), 205), -1, np.int32)
        for b, path in enumerate(paths):
            wide[b, 2:2 + len(path)] = path
        w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], put(wide, dev)[:, 2:202],
                   put(np.array([len(p) for p in paths], np.int32), dev), cu_q=st["cu_q"])
        torch.cuda.synchronize()
        check_keep(batch, paths, st["cache"].cpu().numpy(), st["scale"].cpu().numpy())


def test_keep_odd_paths_and_pages():
    """Counts beyond the nodes, nodes below their place or beyond the sequence,
    absent pages, scale 0, sequences without nodes, more nodes than length."""
    import torch
    dev = device()
    log("keep odd paths")
    batch = Batch([(60, 30), (40, 20), (33, 5), (20, 0), (50, 50), (48, 16)], 16, 2, 64, 15)
    batch.table[1, 2] = -1                           # of nodes 12 and up
    batch.table[4, 0] = batch.pages
    batch.scale[batch.table[0, 2]] = 0
    paths = [[0, 1, 1, 2, 9, 29], [0, 13, 14], [0, 4, 99, -1, 4], [], [0, 20, 30, 31, 40], list(range(16))]
    wide = np.full((6, 20), 3, np.int32)
    for b, path in enumerate(paths):
        wide[b, :len(path)] = path
    st = batch.device(dev)
    count = np.array([6, 3, 5, 4, 5, 16], np.int32)
    w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], put(wide, dev), put(count, dev),
               cu_q=st["cu_q"])
    torch.cuda.synchronize()
    check_keep(batch, paths, st["cache"].cpu().numpy(), st["scale"].cpu().numpy())
    # as many as the path holds, of a sequence that is shorter than its nodes: left alone
    batch.lens[0] = 10
    st = batch.device(dev)
    w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], put(wide, dev),
               put(np.array([1000, 0, -4, 0, 0, 0], np.int32), dev), cu_q=st["cu_q"])
    torch.cuda.synchronize()
    assert (st["cache"].cpu().numpy() == batch.cache).all()
    # without cu_q: one node each, which stays
    batch = Batch([(n, 1) for n in (1, 16, 33)], 16, 1, 32, 16, cu=False)
    st = batch.device(dev)
    w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], put(np.zeros((3, 1), np.int32), dev),
               put(np.ones(3, np.int32), dev))
    torch.cuda.synchronize()
    check_keep(batch, [[0]] * 3, st["cache"].cpu().numpy(), st["scale"].cpu().numpy())


# ------------------------------------------------------------------- graphs
def test_captured_step():
    """Mask, append, attention, confirmation and moves captured in one graph, on
    a stream of their own; each replay with other inputs equals the eager step."""
    import torch
    dev = device()
    log("captured tree step")
    batch = Batch([(40 + 7 * i, 20) for i in range(6)] + [(3000, 20)], 16, 2, 64, 17)
    table = w4.rope_table(3100, 64, device=dev)
    fixed = batch.device(dev)
    inputs = {}

    def fill(seed):
        rng = np.random.default_rng(seed)
        parents, drafted, sampled = draft(batch.spans, rng, 2)
        flat = lambda x: put(np.concatenate([np.asarray(e) for e in x]).astype(np.int32), dev)
        new = {"parents": flat(parents), "drafted": flat(drafted), "sampled": flat(sampled),
               "qkv": put(rng.standard_normal((batch.tokens, 8, 64)).astype(np.float16), dev),
               "cache": put(batch.cache, dev), "scale": put(batch.scale, dev)}
        for name, t in new.items():
            if name in inputs:
                inputs[name].copy_(t)
            else:
                inputs[name] = t

    def step():
        where = (inputs["cache"], inputs["scale"], fixed["block_table"], fixed["seq_lens"])
        mask, positions = w4.tree_mask(inputs["parents"], fixed["seq_lens"], cu_q=fixed["cu_q"], max_q=20)
        q, k, v = inputs["qkv"].split([4, 2, 2], dim=1)
        q = w4.rope_append(q, k, v, table, *where, cu_q=fixed["cu_q"], positions=positions)
        o = w4.tree_attention(q, *where, mask, cu_q=fixed["cu_q"], max_q=20, max_len=3000)
        path, count, tokens, lens = w4.tree_accept(inputs["drafted"], inputs["parents"], inputs["sampled"],
                                                   fixed["seq_lens"], cu_q=fixed["cu_q"], max_q=20)
        w4.kv_keep(*where, path, count, cu_q=fixed["cu_q"])
        return o, path, count, tokens, lens

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        fill(seed)
        eager = [t.clone() for t in step()] + [inputs["cache"].clone(), inputs["scale"].clone()]
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, [*out, inputs["cache"], inputs["scale"]]):
            assert torch.equal(a, b)
        (torch.rand(1000, device=dev) * 2).sum().item()
