"""sample() on the GPU against 64-bit numpy: whole tokens, and their shares to
the rounding of float32."""
import numpy as np
import pytest

import verify_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import device, log

pytestmark = pytest.mark.gpu


def put(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def logits(rows, vocab, rng, dtype, width=2.2):
    x = width * rng.standard_normal((rows, vocab))
    for r in range(rows):
        high = rng.integers(0, vocab, 12)
        x[r, high] += 6 + 2 * rng.exponential(size=12)
    return x.astype(dtype)


def check(x, u, tokens, probs, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Tokens as numpy draws them; shares within half a step of float32 and what
    the weights' rounding to 2^-44 of the largest adds up to: at most 2^-45 for
    each of the row's, of a sum of at least 1."""
    value = lambda v, r: v[r] if np.ndim(v) else v
    for r in range(len(x)):
        want, share = ref.sample(x[r].astype(np.float64), float(u[r]), *(
            float(np.float32(value(v, r))) for v in (temperature,)), int(value(top_k, r)),
            *(float(np.float32(value(v, r))) for v in (top_p, min_p)))
        assert tokens[r] == want, (r, tokens[r], want)
        if want < 0:
            assert np.isnan(probs[r]) == np.isnan(share) and (np.isnan(share) or probs[r] == 0)
        else:
            assert abs(probs[r] - share) <= share * (1.001 * 2.0 ** -24 + x.shape[1] * 2.0 ** -45) + 2.0 ** -150


def run(x, u, dev, **kw):
    import torch
    kw = {k: put(v, dev) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    tokens, probs = w4.sample(x if torch.is_tensor(x) else put(x, dev), put(u, dev), **kw)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), probs.cpu().numpy()


FILTERS = [dict(), dict(temperature=0.7, top_k=50), dict(top_p=0.9), dict(min_p=0.05),
           dict(temperature=1.4, top_k=200, top_p=0.8, min_p=0.01), dict(temperature=0.0), dict(top_k=1),
           dict(top_k=7, top_p=0.5), dict(temperature=3.0, top_p=0.999)]


@pytest.mark.parametrize("filters", FILTERS, ids=str)
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 63, 513, 4097, 32000, 50257, 131072])
def test_sizes_and_filters(vocab, dtype, filters):
    dev = device()
    log(f"sample vocab={vocab} {dtype.__name__} {filters}")
    rng = np.random.default_rng(vocab)
    rows = 9 if vocab < 40000 else 3
    x, u = logits(rows, vocab, rng, dtype), rng.random(rows).astype(np.float32)
    check(x, u, *run(x, u, dev, **filters), **filters)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_rows_at_any_place(dtype, shift):
    """Rows that begin at any element and have any stride."""
    dev = device()
    log(f"sample strides {dtype.__name__} {shift}")
    rng = np.random.default_rng(shift)
    wide = np.full((7, 1000 + shift * 2 + 1), 60000, dtype)      # would be drawn
    wide[:, shift:1000 + shift] = logits(7, 1000, rng, dtype)
    u = rng.random(7).astype(np.float32)
    full = put(wide, dev)
    for part, host in ((full[:, shift:1000 + shift], wide[:, shift:1000 + shift]),
                       (full[::2, shift:shift + 5], wide[::2, shift:shift + 5])):
        for filters in (dict(), dict(top_p=0.7), dict(top_k=3), dict(temperature=0.0)):
            check(host, u[:len(host)], *run(part, u[:len(host)], dev, **filters), **filters)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_ties(dtype):
    """Equal logits: the first ones by number are kept; 0 and -0 are equal."""
    dev = device()
    log(f"sample ties {dtype.__name__}")
    rng = np.random.default_rng(3)
    x = rng.integers(-2, 3, (40, 3001)).astype(dtype)
    x[:20] = np.where(rng.random((20, 3001)) < 0.5, np.copysign(0, -1), 0).astype(dtype)
    x[30:35, ::2] = -np.inf
    u = rng.random(40).astype(np.float32)
    for filters in (dict(), dict(top_k=1000), dict(top_p=0.3), dict(top_k=700, top_p=0.5), dict(min_p=1.0),
                    dict(temperature=0.0), dict(top_k=3000, min_p=0.3, temperature=0.5), dict(top_k=1)):
        check(x, u, *run(x, u, dev, **filters), **filters)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_values_that_are_not_ordinary(dtype):
    dev = device()
    log(f"sample not ordinary {dtype.__name__}")
    rng = np.random.default_rng(4)
    x = logits(14, 777, rng, dtype)
    x[0] = -np.inf
    x[1, 5] = np.nan
    x[2, 776] = np.inf
    x[3] = -np.inf
    x[3, 400] = -3.0                                  # one token left
    x[4, 0] = -np.nan
    x[5, 1:] = -np.inf
    x[6] = np.finfo(dtype).max                        # the largest, all equal
    x[7] = np.finfo(dtype).min
    x[8] = np.linspace(0, 500, 777) * np.finfo(dtype).smallest_subnormal
    x[9, 13] = np.finfo(dtype).max
    x[10, ::3] = -np.inf
    x[11] = np.finfo(dtype).min
    x[11, 9] = np.finfo(dtype).max
    u = rng.random(14).astype(np.float32)
    for filters in FILTERS:
        check(x, u, *run(x, u, dev, **filters), **filters)


def test_extreme_settings():
    """Settings at and beyond the ends of their ranges, and random numbers there:
    the nearest counts."""
    dev = device()
    log("sample extreme settings")
    rng = np.random.default_rng(5)
    x = logits(8, 2000, rng, np.float16)
    u = np.array([0.0, 1 - 2.0 ** -24, 1.0, -1.0, np.nan, 0.5, 7.0, 1e-30], np.float32)
    for filters in (dict(temperature=1e-30), dict(temperature=1e30), dict(temperature=1e-45), dict(top_k=2 ** 40),
                    dict(top_k=-3), dict(top_k=2000), dict(top_k=1999), dict(top_p=0.0), dict(top_p=-1.0),
                    dict(top_p=1e-12), dict(top_p=5.0), dict(top_p=1 - 2.0 ** -24), dict(min_p=-1.0),
                    dict(min_p=2.0), dict(min_p=1e-30)):
        clean = {**filters, "top_k": min(max(filters.get("top_k", 0), 0), 2 ** 31 - 1)}
        check(x, u, *run(x, u, dev, **filters), **clean)
    for bad in (dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
                dict(top_p=float("nan")), dict(min_p=float("nan"))):
        with pytest.raises(w4.W4A8Error):
            run(x, u, dev, **bad)
    # on the device such a setting concerns its row alone
    for name in ("temperature", "top_p", "min_p"):
        each = np.full(8, 0.5, np.float32)
        each[3] = np.nan
        if name == "temperature":
            each[5], each[6] = -1.0, np.inf
        tokens, probs = run(x, u, dev, **{name: each})
        bad = ~np.isfinite(each) | (each < 0)
        assert (tokens[bad] == -1).all() and np.isnan(probs[bad]).all() and (tokens[~bad] >= 0).all()


def test_settings_of_each_row():
    dev = device()
    log("sample settings per row")
    rng = np.random.default_rng(6)
    rows = 300
    x, u = logits(rows, 5000, rng, np.float16), rng.random(rows).astype(np.float32)
    filters = dict(temperature=rng.choice([0.0, 0.5, 1.0, 1.7], rows).astype(np.float32),
                   top_k=rng.choice([0, -1, 1, 40, 6000, 2 ** 31 - 1], rows).astype(np.int32),
                   top_p=rng.choice([0.2, 0.9, 1.0], rows).astype(np.float32),
                   min_p=rng.choice([0.0, 0.02], rows).astype(np.float32))
    check(x, u, *run(x, u, dev, **filters), **filters)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("vocab", [8191, 8192, 20000, 32767, 32768, 70001])
def test_long_rows_of_every_kind(vocab, dtype):
    """Rows that are looked at by several workgroups before: flat ones, whose kept
    tokens are too many to list, steep ones, ties across the bound, few finite
    logits, none, a NaN at an end; with every kind of filter."""
    dev = device()
    log(f"sample long rows {vocab} {dtype.__name__}")
    rng = np.random.default_rng(vocab)
    x = logits(12, vocab, rng, dtype)
    x[0] = (0.01 * rng.standard_normal(vocab)).astype(dtype)
    x[1] = (30 * rng.standard_normal(vocab)).astype(dtype)
    x[2] = rng.integers(0, 3, vocab)
    x[3] = 1.0
    x[4] = -np.inf
    x[4, vocab - 3:] = [1.0, 2.0, 1.5]
    x[5] = -np.inf
    x[6, vocab - 1] = np.nan
    x[7, 0] = np.inf
    x[8, ::2] = -np.inf
    x[9] = np.sort(x[9])
    x[10] = np.sort(x[10])[::-1]
    u = rng.random(12).astype(np.float32)
    for filters in FILTERS + [dict(top_k=600), dict(top_k=513, top_p=0.3), dict(top_k=vocab - 1), dict(min_p=1e-4),
                              dict(min_p=0.5, top_p=0.999), dict(min_p=1.0), dict(top_p=0.5, temperature=20.0),
                              dict(min_p=1e-30, temperature=0.3), dict(top_k=40, min_p=0.2)]:
        check(x, u, *run(x, u, dev, **filters), **filters)
    each = dict(top_k=rng.choice([0, 5, 700], 12).astype(np.int32), top_p=rng.choice([0.7, 1.0], 12).astype(np.float32),
                temperature=rng.choice([0.0, 1.0], 12).astype(np.float32), min_p=rng.choice([0.0, 0.1], 12).astype(np.float32))
    check(x, u, *run(x, u, dev, **each), **each)


def test_the_whole_range_of_u():
    """Every token of a small row is drawn over its share of [0, 1)."""
    dev = device()
    log("sample u")
    x = np.array([[0.0, 1.0, -np.inf, 2.0, -1.0, 0.5]], np.float32)
    u = (np.arange(4096) / 4096).astype(np.float32)
    rows = np.repeat(x, 4096, axis=0)
    tokens, probs = run(rows, u, dev)
    check(rows, u, tokens, probs)
    share = np.exp(x[0].astype(np.float64)) / np.exp(x[0].astype(np.float64)).sum()
    drawn = np.bincount(tokens, minlength=6) / 4096
    assert (np.abs(drawn - share) <= 1 / 4096).all() and (np.diff(tokens) >= 0).all()


def test_largest_vocabulary_many_rows_and_none():
    import torch
    dev = device()
    log("sample largest")
    x = torch.full((3, 1 << 19), 1.0, dtype=torch.float32, device=dev)        # all weights are the largest
    x[1, -1] = 9.0
    u = np.array([0.0, 0.5, 1 - 2.0 ** -24], np.float32)
    tokens, probs = run(x, u, dev)
    check(x.cpu().numpy(), u, tokens, probs)
    assert tokens[0] == 0 and tokens[2] == (1 << 19) - 1
    half = x.half()
    check(half.cpu().numpy(), u, *run(half, u, dev, top_p=0.25), top_p=0.25)
    with pytest.raises(w4.W4A8Error):
        w4.sample(torch.zeros((1, (1 << 19) + 1), dtype=torch.float16, device=dev), put(u[:1], dev))
    tokens, probs = w4.sample(torch.zeros((0, 10), device=dev), put(u[:0], dev))
    assert tokens.shape == (0,) and probs.shape == (0,)
    log("sample many rows")
    rng = np.random.default_rng(7)
    x, u = logits(5000, 33, rng, np.float16), rng.random(5000).astype(np.float32)
    check(x, u, *run(x, u, dev, top_p=0.8), top_p=0.8)


def test_offsets_beyond_32_bits():
    """Rows at byte offsets beyond 2^32."""
    import torch
    dev = device()
    log("sample far rows")
    far = torch.empty(5 * (1 << 29) + 4096, dtype=torch.float16, device=dev)
    x = far.as_strided((6, 4000), ((1 << 29), 1))[:5]
    rng = np.random.default_rng(8)
    host, u = logits(5, 4000, rng, np.float16), rng.random(5).astype(np.float32)
    x.copy_(put(host, dev))
    check(host, u, *run(x, u, dev, top_p=0.9, top_k=100), top_p=0.9, top_k=100)


def test_captured_and_on_two_streams():
    """Captured and replayed with other logits, and two calls at once: each
    equals the eager call alone."""
    import torch
    dev = device()
    log("sample graph")
    rng = np.random.default_rng(9)
    batches = [(logits(20, 40000, rng, np.float16), rng.random(20).astype(np.float32)) for _ in range(4)]
    x, u = put(batches[0][0], dev), put(batches[0][1], dev)
    k = put(rng.integers(0, 60, 20).astype(np.int32), dev)
    alone = [tuple(t.clone() for t in w4.sample(put(a, dev), put(b, dev), 0.8, k, 0.9)) for a, b in batches]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.sample(x, u, 0.8, k, 0.9)
    for (a, b), want in zip(batches, alone):
        x.copy_(put(a, dev))
        u.copy_(put(b, dev))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        (torch.rand(1000, device=dev) * 2).sum().item()
    streams = [torch.cuda.Stream(device=dev) for _ in batches]
    inputs = [(put(a, dev), put(b, dev)) for a, b in batches]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = [w4.sample(a, b, 0.8, k, 0.9, stream=s) for (a, b), s in zip(inputs, streams)]
        torch.cuda.synchronize()
        for got, want in zip(outs, alone):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_groups_than_a_list_holds():
    """Rows of which every 128 bytes hold a token at the bound, and others whose
    few tokens above it are far apart; counts around the largest that maxima bound."""
    dev = device()
    log("sample many groups")
    rng = np.random.default_rng(10)
    vocab = 1 << 19
    for dtype in (np.float16, np.float32):
        x = np.zeros((4, vocab), dtype)
        x[1] = rng.integers(0, 2, vocab)
        x[2] = logits(1, vocab, rng, dtype)[0]
        x[3, ::4099] = 8.0
        u = np.array([0.3, 0.999, 0.6, 0.1], np.float32)
        for filters in (dict(top_k=50), dict(top_k=2048), dict(top_k=2049, top_p=0.9), dict(min_p=0.4),
                        dict(top_k=100, top_p=0.5, temperature=0.3)):
            check(x, u, *run(x, u, dev, **filters), **filters)


def test_long_rows_with_settings_of_each():
    """As for short rows: settings of every row, and at the ends of their ranges."""
    dev = device()
    log("sample long rows, settings per row")
    rng = np.random.default_rng(12)
    rows, vocab = 70, 30001
    x, u = logits(rows, vocab, rng, np.float16), rng.random(rows).astype(np.float32)
    u[:5] = 0.0, 1 - 2.0 ** -24, 1.0, -1.0, np.nan
    filters = dict(temperature=rng.choice([0.0, 0.5, 1.0, 1.7, 1e-30, 1e30], rows).astype(np.float32),
                   top_k=rng.choice([0, 0, -1, 1, 40, 300, 2048, 30000, 30001, 2 ** 31 - 1], rows).astype(np.int32),
                   top_p=rng.choice([0.0, 0.2, 0.9, 1.0, 1 - 2.0 ** -24], rows).astype(np.float32),
                   min_p=rng.choice([0.0, 0.02, 2.0], rows).astype(np.float32))
    check(x, u, *run(x, u, dev, **filters), **filters)
    filters["top_p"][7] = filters["min_p"][8] = filters["temperature"][9] = np.nan
    tokens, probs = run(x, u, dev, **filters)
    assert (tokens[7:10] == -1).all() and np.isnan(probs[7:10]).all()
    assert (np.delete(tokens, [7, 8, 9]) >= 0).all()


def test_long_rows_beyond_32_bits():
    import torch
    dev = device()
    log("sample far long rows")
    far = torch.empty(4 * (1 << 29) + 40960, dtype=torch.float16, device=dev)
    x = far.as_strided((5, 40000), ((1 << 29), 1))
    rng = np.random.default_rng(13)
    host, u = logits(5, 40000, rng, np.float16), rng.random(5).astype(np.float32)
    x.copy_(put(host, dev))
    for filters in (dict(top_p=0.9), dict(top_k=100), dict(min_p=0.1), dict()):
        check(host, u, *run(x, u, dev, **filters), **filters)
