"""rope_append and paged_attention on the GPU against 64-bit numpy."""
import numpy as np
import pytest

import decoder_ref as dref
import w4a8_gemm_amd as w4
from gpu_util import device, log

pytestmark = pytest.mark.gpu


class Batch:
    """Seeded sequences over a shuffled pool: `spans` are (length with the new
    tokens, new tokens) pairs, cu False means one new token each."""

    def __init__(self, spans, page, kv_heads, dim, seed, cu=True, spare=3, wide=0):
        rng = np.random.default_rng(seed)
        self.spans, self.page, self.kv_heads, self.dim = spans, page, kv_heads, dim
        used = [-(-length // page) for length, _ in spans]
        self.pages = sum(used) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        most = max(max(used), 1) + wide
        self.table = np.full((len(spans), most), -1, np.int32)      # unused entries: no page
        done = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[done:done + n]
            done += n
        self.lens = np.array([length for length, _ in spans], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in spans])]).astype(np.int32)
        self.tokens = int(self.cu[-1])
        self.ragged = cu
        assert cu or all(n == 1 for _, n in spans)
        self.cache = rng.integers(-127, 128, (self.pages, 2, kv_heads, page, dim)).astype(np.int8)
        self.scale = (rng.uniform(0.3, 2.5, (self.pages, 2, kv_heads)) / 127).astype(np.float16)
        self.rng = rng

    def device(self, dev):
        import torch
        put = lambda a: torch.from_numpy(a.copy()).to(dev)
        return {"cache": put(self.cache), "scale": put(self.scale), "block_table": put(self.table),
                "seq_lens": put(self.lens), "cu_q": put(self.cu) if self.ragged else None}


def append(batch, dev_state, qkv, heads, cos_sin, interleaved=False, in_place=False):
    """rope_append on the parts of one fused [tokens, heads + 2 kv_heads, dim]
    tensor; returns q, cache, scale as numpy."""
    import torch
    kvh = batch.kv_heads
    q, k, v = qkv.split([heads, kvh, kvh], dim=1)
    st = dev_state
    out = w4.rope_append(q, k, v, cos_sin, st["cache"], st["scale"], st["block_table"], st["seq_lens"],
                         cu_q=st["cu_q"], interleaved=interleaved, out=q if in_place else None)
    torch.cuda.synchronize()
    return out.cpu().numpy(), st["cache"].cpu().numpy(), st["scale"].cpu().numpy()


def check_append(batch, qkv, heads, table, interleaved, q, cache, scale):
    """Every output value against the formula."""
    kvh, page, dim = batch.kv_heads, batch.page, batch.dim
    half = table.shape[1] // 2 if table is not None else 0
    touched = np.zeros(batch.cache.shape[:1] + (page,), bool)        # slots written or rescaled
    for b, (length, n) in enumerate(batch.spans):
        lo = batch.cu[b]
        turned = qkv[lo:lo + n].astype(np.float64)
        for i in range(n if half else 0):
            pos = min(length - n + i, table.shape[0] - 1)
            turned[i, :heads + kvh] = dref.rotate(qkv[lo + i, :heads + kvh], pos, table, interleaved)
        # two products and a sum in fp32 of values up to |x|: then one rounding to fp16
        slack = 4 * 2.0 ** -24 * np.abs(qkv[lo:lo + n].astype(np.float64)).max(axis=2, keepdims=True) * 2
        want_q = turned[:, :heads]
        assert (np.abs(q[lo:lo + n] - want_q) <= dref.half_ulp16(want_q) * 1.001 + slack[:, :heads]).all()
        for idx in range((length - n) // page, -(-length // page)):
            begin, end = max(length - n, idx * page), min(length, (idx + 1) * page)
            at = int(batch.table[b, idx])
            if begin >= end or not 0 <= at < batch.pages:
                continue
            first = begin - idx * page
            touched[at, :first + end - begin] = True
            new = turned[begin - (length - n):end - (length - n), heads:].reshape(-1, 2, kvh, dim)
            new_slack = slack[begin - (length - n):end - (length - n), heads:].reshape(-1, 2, kvh, 1)
            for w in range(2):
                for h in range(kvh):
                    s = float(scale[at, w, h])
                    old = float(batch.scale[at, w, h]) if first else 0.0
                    amax, err = np.abs(new[:, w, h]).max(), new_slack[:, w, h].max()
                    own = amax / 127
                    if s != old:                     # grew: the fp16 nearest to amax / 127
                        assert s > old
                        assert abs(s - own) <= dref.half_ulp16(own) * 1.001 + err / 127 + own * 2.0 ** -23
                    else:                            # or stayed, because amax / 127 rounds to no more
                        assert own <= old + dref.half_ulp16(own) * 1.001 + err / 127 + own * 2.0 ** -23
                    codes = cache[at, w, h].astype(np.float64)
                    held = batch.cache[at, w, h, :first].astype(np.float64)
                    if s == old:
                        assert (codes[:first] == held).all()
                    elif first:
                        assert (np.abs(codes[:first] - held * old / s) <= 0.5 + 127 * 2.0 ** -22).all()
                    want = np.clip(new[:, w, h] / s, -127, 127) if s else np.zeros_like(new[:, w, h])
                    tol = 0.5 + 127.5 * 4 * 2.0 ** -24 + (err / s if s else 0)
                    assert (np.abs(codes[first:first + end - begin] - want) <= tol).all()
    same = ~touched
    assert (cache.transpose(0, 3, 1, 2, 4)[same] == batch.cache.transpose(0, 3, 1, 2, 4)[same]).all()
    untouched = ~touched.any(axis=1)
    assert (scale[untouched].view(np.uint16) == batch.scale[untouched].view(np.uint16)).all()


def rope(positions, rotary, dev):
    return w4.rope_table(positions, rotary, device=dev) if rotary else None


RAGGED = [(70, 70), (5, 1), (200, 33), (64, 0), (0, 0), (17, 17), (129, 2), (128, 64)]


@pytest.mark.parametrize("spans,page,heads,kv_heads,dim,rotary,interleaved,cu", [
    (RAGGED, 16, 8, 2, 128, 128, False, True),
    (RAGGED, 64, 8, 2, 128, 128, True, True),
    (RAGGED, 128, 5, 5, 64, 32, False, True),
    (RAGGED, 32, 6, 3, 80, 48, True, True),
    (RAGGED, 16, 3, 1, 256, 256, False, True),
    (RAGGED, 1024, 4, 2, 16, 16, False, True),
    (RAGGED, 32, 7, 1, 96, 0, False, True),
    ([(1, 1)], 16, 4, 4, 128, 128, False, False),
    ([(n, 1) for n in (1, 16, 17, 31, 32, 33, 100)], 16, 32, 8, 128, 128, False, False),
    ([(n, 1) for n in (64, 65, 2, 128)], 64, 12, 4, 64, 64, True, False),
    ([(n, n) for n in (300, 1, 513)], 64, 9, 3, 192, 64, False, True),
])
def test_append(spans, page, heads, kv_heads, dim, rotary, interleaved, cu):
    import torch
    dev = device()
    log(f"append page={page} heads={heads}/{kv_heads} dim={dim} rotary={rotary} cu={cu}")
    batch = Batch(spans, page, kv_heads, dim, 1, cu=cu, wide=1)
    qkv = batch.rng.standard_normal((batch.tokens, heads + 2 * kv_heads, dim)).astype(np.float16)
    table = rope(256 if max(n for n, _ in spans) < 256 else 600, rotary, dev)
    st = batch.device(dev)
    got = append(batch, st, torch.from_numpy(qkv).to(dev), heads, table, interleaved)
    check_append(batch, qkv, heads, table.cpu().numpy() if rotary else None, interleaved, *got)


@pytest.mark.parametrize("size", [0.01, 1.0, 30.0])
def test_append_growth_of_the_scale(size):
    """One token after another: none, some and every one of them raises its
    page's scale; codes before it follow."""
    import torch
    dev = device()
    log(f"append growth size={size}")
    batch = Batch([(20, 1), (33, 1), (48, 1), (7, 1)], 16, 2, 128, 2, cu=False)
    for step in range(4):
        qkv = (batch.rng.standard_normal((4, 4 + 4, 128)) * size * (1 + step)).astype(np.float16)
        st = batch.device(dev)
        q, cache, scale = append(batch, st, torch.from_numpy(qkv).to(dev), 4, None)
        check_append(batch, qkv, 4, None, False, q, cache, scale)
        batch.cache, batch.scale = cache, scale


def test_append_in_place_and_zero_tokens():
    """q rotated over itself; a block of zeros has scale 0 and codes 0."""
    import torch
    dev = device()
    log("append in place, zeros")
    batch = Batch([(40, 40), (16, 16)], 16, 2, 64, 3)
    qkv = batch.rng.standard_normal((56, 4 + 4, 64)).astype(np.float16)
    qkv[40:] = 0
    table = rope(64, 64, dev)
    st = batch.device(dev)
    got = append(batch, st, torch.from_numpy(qkv).to(dev), 4, table, in_place=True)
    check_append(batch, qkv, 4, table.cpu().numpy(), False, *got)
    at = batch.table[1, 0]
    assert (got[1][at] == 0).all() and (got[2][at] == 0).all()


def test_append_positions_beyond_the_table_and_absent_pages():
    """Positions past the table's end take its last row; pages the block table
    does not have are not written."""
    import torch
    dev = device()
    log("append clamps")
    batch = Batch([(60, 60), (50, 20)], 16, 1, 64, 4)
    batch.table[0, 1] = -1
    batch.table[1, 3] = batch.pages
    qkv = batch.rng.standard_normal((80, 2 + 2, 64)).astype(np.float16)
    table = rope(45, 64, dev)
    st = batch.device(dev)
    got = append(batch, st, torch.from_numpy(qkv).to(dev), 2, table)
    check_append(batch, qkv, 2, table.cpu().numpy(), False, *got)


def test_append_marks_a_block_that_is_not_finite():
    """NaN in one key head: that block's scale alone; infinity likewise."""
    import torch
    dev = device()
    log("append non-finite")
    batch = Batch([(32, 32)], 32, 4, 64, 5)
    qkv = batch.rng.standard_normal((32, 4 + 8, 64)).astype(np.float16)
    qkv[7, 4 + 1, 3] = np.nan                 # key head 1
    qkv[9, 8 + 2, 3] = -np.inf                # value head 2
    st = batch.device(dev)
    _, _, scale = append(batch, st, torch.from_numpy(qkv).to(dev), 4, None)
    at = batch.table[0, 0]
    assert np.isnan(scale[at, 0, 1]) and np.isinf(scale[at, 1, 2])
    finite = np.isfinite(scale[at])
    assert finite.sum() == 6 and not finite[0, 1] and not finite[1, 2]


# ----------------------------------------------------------------- attention
def attend(batch, q, dev, window=0, state=None, **kw):
    import torch
    st = state or batch.device(dev)
    o = w4.paged_attention(torch.from_numpy(q).to(dev), st["cache"], st["scale"], st["block_table"],
                           st["seq_lens"], cu_q=st["cu_q"], window=window, **kw)
    torch.cuda.synchronize()
    return o.cpu().numpy()


def check_attention(batch, q, o, window=0, scale=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, bound = dref.attention(q, batch.cache, batch.scale, batch.table, batch.lens, batch.cu, scale, window)
    err = np.abs(o.astype(np.float64) - want)
    assert (err <= bound).all(), (np.unravel_index((err - bound).argmax(), err.shape), (err / bound).max())


DECODE = [(n, 1) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 500)]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64), (7, 1, 80), (20, 1, 128),
                                                (16, 2, 256), (3, 3, 16), (40, 1, 48), (2, 1, 192)])
def test_decode(page, heads, kv_heads, dim):
    dev = device()
    log(f"decode page={page} heads={heads}/{kv_heads} dim={dim}")
    batch = Batch(DECODE, page, kv_heads, dim, 6, cu=False)
    q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
    check_attention(batch, q, attend(batch, q, dev))


@pytest.mark.parametrize("length", [255, 512, 1000, 4097, 9000])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (2, 2, 64), (6, 1, 256)])
def test_decode_split_over_a_long_sequence(length, heads, kv_heads, dim):
    """Few rows: the keys are split over workgroups and joined, also where
    the sequence is far shorter or longer than max_len said."""
    dev = device()
    for bound in (None, 64, length, 20 * length):
        log(f"decode long={length} heads={heads}/{kv_heads} dim={dim} max_len={bound}")
        batch = Batch([(length, 1), (3, 1)], 64, kv_heads, dim, 7, cu=False, wide=40)
        q = (2 * batch.rng.standard_normal((2, heads, dim))).astype(np.float16)
        check_attention(batch, q, attend(batch, q, dev, max_len=bound))


CHUNKS = [(70, 70), (5, 1), (200, 33), (64, 0), (0, 0), (17, 17), (129, 2), (300, 64), (1, 1), (257, 130)]


@pytest.mark.parametrize("window", [0, 1, 40, 1000])
@pytest.mark.parametrize("page,heads,kv_heads,dim", [(16, 8, 2, 128), (64, 4, 4, 64), (32, 6, 2, 80),
                                                     (128, 5, 1, 256), (16, 17, 1, 96), (64, 32, 1, 128)])
def test_chunks(page, heads, kv_heads, dim, window):
    """Chunks of new tokens of every kind in one batch: whole prompts, single
    tokens, none, ragged ends, after earlier tokens or not."""
    dev = device()
    log(f"chunks page={page} heads={heads}/{kv_heads} dim={dim} window={window}")
    batch = Batch(CHUNKS, page, kv_heads, dim, 8)
    q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
    check_attention(batch, q, attend(batch, q, dev, window=window), window)
    # a bound on the new tokens that is too small changes nothing but the time
    check_attention(batch, q, attend(batch, q, dev, window=window, max_q=1, max_len=10), window)


@pytest.mark.parametrize("dim,window", [(128, 0), (128, 100), (80, 0)])
def test_chunks_that_fill_the_device(dim, window):
    """So many row tiles that the kernel with two halves of waves is taken."""
    dev = device()
    log(f"wide tiles dim={dim} window={window}")
    spans = [(300, 300), (5, 1), (330, 33), (0, 0), (257, 257), (129, 2), (64, 64), (90, 17)]
    batch = Batch(spans, 16, 64, dim, 18)
    q = (2 * batch.rng.standard_normal((batch.tokens, 128, dim))).astype(np.float16)
    check_attention(batch, q, attend(batch, q, dev, window=window), window)


@pytest.mark.parametrize("length,new,heads,kv_heads,dim,window", [
    (3000, 30, 8, 1, 128, 0), (2500, 64, 4, 2, 64, 0), (1700, 9, 20, 1, 256, 0), (4000, 50, 4, 1, 96, 1500)])
def test_chunk_over_a_long_sequence(length, new, heads, kv_heads, dim, window):
    """Many rows a tile and few tiles: their keys are split and joined."""
    dev = device()
    log(f"chunk over a long sequence len={length} new={new} heads={heads}/{kv_heads} dim={dim}")
    batch = Batch([(length, new), (20, 20)], 32, kv_heads, dim, 19)
    q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
    for bound in (None, length // 2):
        check_attention(batch, q, attend(batch, q, dev, window=window, max_len=bound), window)


@pytest.mark.parametrize("heads,kv_heads,dim", [(20, 1, 64), (20, 1, 128), (34, 2, 96), (18, 1, 256), (68, 4, 32)])
@pytest.mark.parametrize("window", [0, 150])
def test_tiles_with_waves_that_have_no_rows(heads, kv_heads, dim, window):
    """One wave of four makes scores of the first key tile, the others go
    straight to staging later tiles' keys; or, under a window, waves start at
    different tiles.  Every tile's keys are of another size, so that keys of
    a later tile in the place of an earlier one's would show."""
    dev = device()
    spans = [(n, 1) for n in (20, 64, 65, 129, 193, 257, 400, 640, 90, 310)] + [(500, 9), (330, 40), (260, 13)]
    for cu in (True, False):
        log(f"waves without rows heads={heads}/{kv_heads} dim={dim} window={window} cu={cu}")
        batch = Batch(spans if cu else spans[:10], 16, kv_heads, dim, 22, cu=cu)
        for b in range(len(batch.spans)):
            for i, at in enumerate(batch.table[b]):
                if at >= 0:
                    batch.scale[at, 0] *= np.float16((1.0, 0.25, 3.0)[i // 4 % 3])
        q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
        # unsplit, and split over the keys
        check_attention(batch, q, attend(batch, q, dev, window=window, max_q=40, max_len=64), window)
        check_attention(batch, q, attend(batch, q, dev, window=window, max_q=40, max_len=4096), window)


@pytest.mark.parametrize("light", [0.0, 2.0 ** -24, 2.0 ** -12])
@pytest.mark.parametrize("spans,heads,kv_heads,dim,cu", [
    ([(600, 1), (600, 1), (70, 1)], 8, 2, 128, False),                  # one row tile of 16
    ([(600, 40), (600, 64), (70, 9)], 8, 2, 128, True),                 # 4 waves
    ([(600, 40), (600, 64), (70, 9)], 4, 2, 64, True),
    ([(600, 40), (600, 17), (70, 9)], 4, 2, 256, True),
    ([(600, 300), (400, 300), (300, 257), (64, 17)], 128, 64, 128, True),   # 8 waves
])
def test_mass_in_pages_of_small_values(spans, heads, kv_heads, dim, cu, light):
    """One key of large values, at score 0, beside hundreds at score -8 whose
    pages' values are 0 or tiny: these carry a sixth of the softmax's sum,
    but, with the value scale in it, less than 2^-24 of the largest weight.

    Beyond the reference's bound, such a weight is rounded at fp16's smallest
    steps: the largest weight is at least 2^10 there, half a step is 2^-25, so a
    key's product is off by 2^-35 * 127 of the largest weight."""
    dev = device()
    log(f"small values heads={heads}/{kv_heads} dim={dim} light={light}")
    page = 16
    batch = Batch(spans, page, kv_heads, dim, 23, cu=cu)
    # score of a key: the mean of the query's values, times code * scale
    batch.cache[:, 0] = -100
    batch.scale[:, 0] = 0.08
    batch.scale[:, 1] = light
    if light == 0:
        batch.cache[:, 1] = 0
    for b, (length, _) in enumerate(spans):
        at = batch.table[b, 0 if b % 2 == 0 else (length // 2) // page]   # before and after most others
        batch.scale[at, 0], batch.scale[at, 1] = 0.3, 1.0
        batch.cache[at, 0, :, 5] = 0
        batch.cache[at, 1] = batch.rng.integers(64, 128, batch.cache[at, 1].shape)
    q = np.broadcast_to(batch.rng.choice([0.75, 1.0, 1.25], (batch.tokens, heads, 1)), (batch.tokens, heads, dim))
    q = q.astype(np.float16)
    o = attend(batch, q, dev, scale=1.0 / dim)
    want, bound = dref.attention(q, batch.cache, batch.scale, batch.table, batch.lens, batch.cu, 1.0 / dim)
    err = np.abs(o.astype(np.float64) - want)
    bound = bound + 600 * 127 * 2.0 ** -35
    assert (err <= bound).all(), (np.unravel_index((err - bound).argmax(), err.shape), (err / bound).max())


def test_many_rows_joined():
    """More split rows than the join takes four waves each for."""
    dev = device()
    log("many split rows")
    lens = np.random.default_rng(20).integers(1, 1500, 80)
    batch = Batch([(int(n), 1) for n in lens], 64, 1, 64, 21, cu=False)
    q = (2 * batch.rng.standard_normal((80, 64, 64))).astype(np.float16)
    check_attention(batch, q, attend(batch, q, dev))


def test_rows_that_see_nothing():
    """Length 0, and every page of a sequence absent: zeros, not NaN."""
    dev = device()
    log("empty rows")
    batch = Batch([(40, 1), (0, 1), (40, 1)], 16, 2, 128, 9, cu=False)
    batch.table[2] = -1
    q = batch.rng.standard_normal((3, 4, 128)).astype(np.float16)
    o = attend(batch, q, dev)
    check_attention(batch, q, o)
    assert (o[1] == 0).all() and (o[2] == 0).all() and (o[0] != 0).any()
    # the same among chunks: more new tokens than the length says
    batch = Batch([(30, 30), (20, 20)], 16, 2, 128, 10)
    batch.lens[1] = 4
    q = batch.rng.standard_normal((50, 4, 128)).astype(np.float16)
    o = attend(batch, q, dev)
    check_attention(batch, q, o)
    assert (o[30:46] == 0).all()


def test_absent_pages_are_not_seen():
    dev = device()
    log("absent pages")
    batch = Batch([(100, 1), (90, 60)], 16, 2, 64, 11)
    batch.table[0, 2] = -1
    batch.table[0, 3] = 10 ** 6
    batch.table[1, 0] = -5
    q = batch.rng.standard_normal((61, 4, 64)).astype(np.float16)
    check_attention(batch, q, attend(batch, q, dev))


@pytest.mark.parametrize("spans,heads,kv_heads,dim,cu", [
    ([(1, 1), (2, 1), (40, 1)], 8, 2, 128, False), ([(3, 3), (200, 70), (30, 30)], 6, 2, 64, True),
    ([(3, 3), (200, 70), (30, 30)], 6, 2, 128, True), ([(3, 3), (200, 70), (30, 30)], 6, 2, 256, True)])
def test_queries_that_are_not_finite(spans, heads, kv_heads, dim, cu):
    """A query head that holds a NaN or an infinity is NaN for every row, also
    where all the scores that it sees are minus infinity; its neighbours stay
    within their bound (their roundings may move: the 32 or 16 rows of a wave move
    their running maxima together)."""
    dev = device()
    log(f"queries that are not finite heads={heads}/{kv_heads} dim={dim}")
    batch = Batch(spans, 16, kv_heads, dim, 27, cu=cu)
    q = batch.rng.standard_normal((batch.tokens, heads, dim)).astype(np.float16)
    want, bound = dref.attention(q, batch.cache, batch.scale, batch.table, batch.lens, batch.cu, dim ** -0.5)
    good = np.ones(heads, bool)
    good[[1, 2, 4]] = False
    q[:, 1, 7], q[:, 2, 5], q[:, 4, 0] = np.nan, np.inf, -np.inf
    o = attend(batch, q, dev)
    assert np.isnan(o[:, ~good]).all()
    assert (np.abs(o.astype(np.float64) - want)[:, good] <= bound[:, good]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_that_are_not_finite_over_absent_pages(dim):
    """A row that sees no key is 0 whatever its query holds; one that sees a
    key is NaN."""
    dev = device()
    log(f"queries that are not finite over absent pages dim={dim}")
    batch = Batch([(200, 40), (200, 40), (90, 1), (90, 1)], 16, 2, dim, 26)
    batch.table[0] = -1
    batch.table[2] = -1
    batch.table[1, :12] = -1                       # positions below 192: its last 8 rows see the rest
    q = batch.rng.standard_normal((82, 4, dim)).astype(np.float16)
    q[:, 1], q[:, 2, 5] = np.nan, np.inf
    o = attend(batch, q, dev)
    assert (o[:72] == 0).all() and (o[80] == 0).all()
    assert np.isnan(o[72:80, 1:3]).all() and np.isnan(o[81, 1:3]).all()
    good = q.copy()
    good[:, 1:3] = 0
    want, bound = dref.attention(good, batch.cache, batch.scale, batch.table, batch.lens, batch.cu, dim ** -0.5)
    assert (np.abs(o - want)[:, ::3] <= bound[:, ::3]).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_nothing_leaks_from_masked_pages(bad):
    """Scales that are NaN or infinite in pages a row does not see (later
    tokens, before the window, pages of no sequence) leave it as it is, in
    every kernel and split."""
    dev = device()
    log(f"masked pages with {bad}")
    page = 16
    batch = Batch([(128, 128), (400, 1)], page, 1, 128, 12)
    q = batch.rng.standard_normal((129, 4, 128)).astype(np.float16)
    clean = attend(batch, q, dev, window=100)
    used = set(batch.table[batch.table >= 0].tolist())
    for p in range(batch.pages):
        if p not in used:
            batch.scale[p] = bad
    batch.scale[batch.table[0, 7]] = bad                      # positions 112 ..
    for i in range(12):                                       # before the second one's window
        batch.scale[batch.table[1, i]] = bad
    o = attend(batch, q, dev, window=100)
    assert np.array_equal(o[:112].view(np.uint16), clean[:112].view(np.uint16))
    assert np.array_equal(o[128].view(np.uint16), clean[128].view(np.uint16))
    assert np.isnan(o[112:128]).all()


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("spans,heads,kv_heads,dim,cu", [
    ([(90, 1), (90, 1), (2000, 1)], 8, 2, 128, False), ([(90, 1), (90, 9), (90, 70)], 16, 1, 128, True),
    ([(90, 1), (90, 9), (90, 70)], 8, 2, 64, True), ([(90, 1), (90, 9), (90, 70)], 20, 1, 256, True),
    ([(90, 90), (300, 300), (280, 257), (70, 70), (90, 40)], 128, 64, 128, True)])
def test_a_key_scale_that_is_not_finite_is_seen(spans, heads, kv_heads, dim, cu, bad):
    """Keys of a block whose scale is infinite or NaN make the rows that see
    them NaN whatever the sign of their codes' product with the query, and
    leave other sequences and other heads as they are."""
    dev = device()
    log(f"key scale {bad} heads={heads}/{kv_heads} dim={dim}")
    batch = Batch(spans, 16, kv_heads, dim, 24, cu=cu)
    q = batch.rng.standard_normal((batch.tokens, heads, dim)).astype(np.float16)
    clean = attend(batch, q, dev)
    batch.scale[batch.table[1, 2], 0, -1] = bad               # positions 32 .. 47, keys of the last kv head
    o = attend(batch, q, dev)
    hit = np.zeros(o.shape[:2], bool)
    length, new = spans[1]
    pos = np.arange(length - new, length)
    hit[batch.cu[1]:batch.cu[2], -(heads // kv_heads):] = (pos >= 32)[:, None]
    assert hit.any() and np.isnan(o[hit]).all()
    assert np.array_equal(o[~hit].view(np.uint16), clean[~hit].view(np.uint16))


@pytest.mark.parametrize("spans,heads,kv_heads,dim,cu", [
    ([(90, 1), (17, 1), (3000, 1)], 8, 2, 128, False), ([(90, 1), (90, 9), (90, 70)], 20, 1, 128, True)])
def test_value_scale_zero_means_values_of_zero(spans, heads, kv_heads, dim, cu):
    """A value is code * scale: codes under a value scale of 0 (a pool that was
    not filled by rope_append) add nothing, and count in the softmax's sum."""
    dev = device()
    log(f"value scale 0 heads={heads}/{kv_heads} dim={dim}")
    batch = Batch(spans, 16, kv_heads, dim, 25, cu=cu)
    q = batch.rng.standard_normal((batch.tokens, heads, dim)).astype(np.float16)
    batch.scale[:, 1] = 0
    o = attend(batch, q, dev)
    assert (o == 0).all()
    # beside pages whose values are tiny as well
    batch.scale[::2, 1] = 2.0 ** -24
    batch.scale[1::4, 1] = np.float16(-0.0)
    check_attention(batch, q, attend(batch, q, dev))


@pytest.mark.parametrize("size", [3e8, -3e8, 1e20, -1e32, 1e34])
@pytest.mark.parametrize("spans,heads,kv_heads,dim,cu", [
    ([(40, 1), (2000, 1)], 8, 2, 128, False), ([(40, 9), (100, 30)], 8, 1, 128, True), ([(40, 9), (100, 30)], 8, 1, 64, True)])
def test_scores_of_any_finite_size(spans, heads, kv_heads, dim, cu, size):
    """Scores of +-1e8 to +-1e34, whose fp32 spacing is 8 or more: the largest one's key alone is left.  Its
    value passes a reciprocal and three products in fp32."""
    dev = device()
    log(f"scores of {size} heads={heads}/{kv_heads} dim={dim}")
    batch = Batch(spans, 16, kv_heads, dim, 28, cu=cu)
    batch.scale[:, 0] = 0.01
    for others, largest in ((-50, -40), (50, 60)):
        batch.cache[:, 0] = others if size > 0 else -others
        for b in range(len(spans)):                # at position 3, where every row sees it
            batch.cache[batch.table[b, 0], 0, :, 3] = largest if size > 0 else -largest
        q = np.full((batch.tokens, heads, dim), 1.0, np.float16)
        o = attend(batch, q, dev, scale=size / dim).astype(np.float64)
        for b in range(len(spans)):
            at = batch.table[b, 0]
            v = batch.cache[at, 1, :, 3].astype(np.float64) * batch.scale[at, 1].astype(np.float64)[:, None]
            v = np.repeat(v, heads // kv_heads, axis=0)
            rows = o[batch.cu[b]:batch.cu[b + 1]]
            assert (np.abs(rows - v) <= dref.half_ulp16(v) * 1.001 + np.abs(v) * 2.0 ** -20).all()


def test_scores_far_apart_and_scales_far_apart():
    """One key holds all the weight, pages whose value scales differ by 2^20,
    pages of zeros, and a score scale of 0 (a plain mean)."""
    dev = device()
    log("extremes")
    batch = Batch([(200, 1), (300, 40)], 16, 2, 128, 13)
    batch.scale[::2, 1] *= np.float16(2.0 ** -10)
    batch.scale[1::2, 1] *= np.float16(2.0 ** 10)
    batch.scale[batch.table[0, 3]] = 0
    batch.cache[batch.table[0, 3]] = 0
    q = (40 * batch.rng.standard_normal((41, 4, 128))).astype(np.float16)
    check_attention(batch, q, attend(batch, q, dev))
    check_attention(batch, q, attend(batch, q, dev, scale=0.0), scale=0.0)
    check_attention(batch, q, attend(batch, q, dev, scale=-0.05), scale=-0.05)


def test_strided_pool_and_rows():
    """Two layers' pages in one allocation, q and o inside wider rows."""
    import torch
    dev = device()
    log("strided pool")
    heads, kvh, dim, page = 8, 2, 64, 32
    batch = Batch(CHUNKS, page, kvh, dim, 14)
    st = batch.device(dev)
    pool = torch.zeros((batch.pages, 2, 2, kvh, page, dim), dtype=torch.int8, device=dev)
    scales = torch.zeros((batch.pages, 2, 2, kvh), dtype=torch.float16, device=dev)
    pool[:, 1], scales[:, 1] = st["cache"], st["scale"]
    st["cache"], st["scale"] = pool[:, 1], scales[:, 1]
    q = batch.rng.standard_normal((batch.tokens, heads, dim)).astype(np.float16)
    wide = torch.zeros((batch.tokens, heads + 4, dim), dtype=torch.float16, device=dev)
    wide[:, :heads] = torch.from_numpy(q).to(dev)
    out = torch.full((batch.tokens, heads + 2, dim), 3.0, dtype=torch.float16, device=dev)
    w4.paged_attention(wide[:, :heads], st["cache"], st["scale"], st["block_table"], st["seq_lens"],
                       cu_q=st["cu_q"], out=out[:, :heads])
    torch.cuda.synchronize()
    check_attention(batch, q, out[:, :heads].cpu().numpy())
    assert (out[:, heads:] == 3.0).all()
    qkv = batch.rng.standard_normal((batch.tokens, heads + 2 * kvh, dim)).astype(np.float16)
    got = append(batch, st, torch.from_numpy(qkv).to(dev), heads, None)
    check_append(batch, qkv, heads, None, False, *got)
    assert (pool[:, 0] == 0).all() and (scales[:, 0] == 0).all()


def test_pages_beyond_2_gib():
    """Pages whose offset passes 2^31 and 2^32 bytes, written and read."""
    import torch
    dev = device()
    log("pool of more than 4 GiB")
    kvh, dim, page, heads = 8, 128, 1024, 16
    pages = (1 << 32) // (2 * kvh * dim * page) + 8
    cache = torch.zeros((pages, 2, kvh, page, dim), dtype=torch.int8, device=dev)
    scale = torch.zeros((pages, 2, kvh), dtype=torch.float16, device=dev)
    batch = Batch([(1500, 1500)], page, kvh, dim, 15)
    far = [pages - 2, pages // 2 + 3]
    qkv = batch.rng.standard_normal((1500, heads + 2 * kvh, dim)).astype(np.float16)
    st = batch.device(dev)
    st["cache"], st["scale"] = cache, scale
    st["block_table"] = torch.tensor([far], dtype=torch.int32, device=dev)
    q, k, v = torch.from_numpy(qkv).to(dev).split([heads, kvh, kvh], dim=1)
    args = (st["cache"], st["scale"], st["block_table"], st["seq_lens"])
    w4.rope_append(q, k, v, None, *args, cu_q=st["cu_q"])
    torch.cuda.synchronize()
    # the same codes in a small pool
    batch.cache = cache[far].cpu().numpy()
    batch.scale = scale[far].cpu().numpy()
    batch.table, batch.pages = np.array([[0, 1]], np.int32), 2
    code = batch.cache.astype(np.float64) * batch.scale.astype(np.float64)[..., None, None]
    back = code[:, 1].transpose(0, 2, 1, 3).reshape(-1, kvh, dim)[:1500]
    assert (np.abs(back - qkv[:, heads + kvh:]) <= 0.51 * batch.scale[:, 1].max()).all()
    last = torch.from_numpy(qkv[-3:, :heads].copy()).to(dev)
    o = w4.paged_attention(last, *args, cu_q=torch.tensor([0, 3], dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    batch.spans, batch.cu = [(1500, 3)], np.array([0, 3], np.int32)
    check_attention(batch, qkv[-3:, :heads], o.cpu().numpy())
    del cache


def test_graph_replays_and_streams():
    """append + attention captured in a graph, replayed with other work between,
    and run on a stream of its own: the same bits as the eager call."""
    import torch
    dev = device()
    log("graph and stream")
    heads, kvh, dim = 8, 2, 128
    batch = Batch([(700, 1), (40, 1), (1, 1)], 16, kvh, dim, 16, cu=False)
    st = batch.device(dev)
    qkv = torch.from_numpy(batch.rng.standard_normal((3, heads + 2 * kvh, dim)).astype(np.float16)).to(dev)
    q, k, v = qkv.split([heads, kvh, kvh], dim=1)
    table = rope(1024, dim, dev)
    turned = torch.empty((3, heads, dim), dtype=torch.float16, device=dev)
    o = torch.empty_like(turned)
    args = (st["cache"], st["scale"], st["block_table"], st["seq_lens"])
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=dev)

    def step(stream=None):
        w4.rope_append(q, k, v, table, *args, out=turned, stream=stream)
        w4.paged_attention(turned, *args, max_len=1024, out=o, workspace=ws, stream=stream)

    step()
    torch.cuda.synchronize()
    want, want_cache = o.clone(), st["cache"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        o.zero_()
        turned.zero_()
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        log(f"replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(st["cache"], want_cache)
    s = torch.cuda.Stream(device=dev)
    o.zero_()
    torch.cuda.synchronize()
    step(stream=s)
    s.synchronize()
    assert torch.equal(o, want)


def test_refusals():
    import torch
    dev = device()
    batch = Batch([(40, 1), (30, 1)], 16, 2, 64, 17, cu=False)
    st = batch.device(dev)
    args = (st["cache"], st["scale"], st["block_table"], st["seq_lens"])
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device=dev)
    k = torch.zeros((2, 2, 64), dtype=torch.float16, device=dev)
    table = rope(64, 64, dev)
    for bad in (lambda: w4.paged_attention(q.float(), *args),
                lambda: w4.paged_attention(q[:1], *args),
                lambda: w4.paged_attention(q[:, :, :32], *args),
                lambda: w4.paged_attention(q.transpose(0, 1), *args),
                lambda: w4.paged_attention(q, args[0].half(), *args[1:]),
                lambda: w4.paged_attention(q, args[0], args[1][:, :1], *args[2:]),
                lambda: w4.paged_attention(q, *args[:2], args[2].long(), args[3]),
                lambda: w4.paged_attention(q, *args[:3], args[3][:1]),
                lambda: w4.paged_attention(q, *args, cu_q=st["seq_lens"]),
                lambda: w4.rope_append(q, k[:1], k, table, *args),
                lambda: w4.rope_append(q, k, k, table.half(), *args),
                lambda: w4.rope_append(q, k, k, table, *args, out=q[:1])):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: w4.paged_attention(q[:, :3].contiguous(), *args), 2),
                        (lambda: w4.paged_attention(q, *args, window=-1), 1),
                        (lambda: w4.paged_attention(q, *args, scale=float("nan")), 1),
                        (lambda: w4.rope_append(q, k, k, rope(64, 8, dev), *args), 2),
                        (lambda: w4.rope_append(q, k, k, rope(64, 128, dev), *args), 1)):
        with pytest.raises(w4.W4A8Error) as err:
            bad()
        assert err.value.status == status
    # nothing to do is no error
    none = torch.zeros((0, 4, 64), dtype=torch.float16, device=dev)
    cu = torch.zeros(3, dtype=torch.int32, device=dev)
    assert w4.paged_attention(none, *args, cu_q=cu).shape == (0, 4, 64)
