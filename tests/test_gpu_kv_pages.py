"""Pages of the cache on the GPU against plain Python: rows that continue others,
fresh pages and copies, pages in use moved together.  Whole numbers: equal."""
import numpy as np
import pytest

import verify_ref as ref
import w4a8_gemm_amd as w4
from gpu_util import device, log

pytestmark = pytest.mark.gpu


def put(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def host(ts):
    import torch
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in ts]


def pool(rows, width, pages, page, rng, shared=0.3, spare=0.2, pins=0.1):
    """Tables over a pool: (table, lens, refs).  Rows share pages of earlier ones
    at their beginning, some hold pages beyond their tokens, some pages are held
    elsewhere, some entries beyond name nothing at all."""
    free = rng.permutation(pages).tolist()
    table, lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    for b in range(rows):
        used = int(rng.integers(0, width + 1))
        first = []
        if b and rng.random() < shared:
            other = int(rng.integers(b))
            full = -(-int(lens[other]) // page)
            first = table[other, :int(rng.integers(0, full + 1))].tolist()
            if any(p < 0 for p in first):
                first = []
        used = min(max(used, len(first)), len(first) + len(free))
        line = first + [free.pop() for _ in range(used - len(first))]
        table[b, :used] = line
        lens[b] = int(rng.integers(max(0, used - 1) * page, used * page + 1)) if used else 0
        if len(first) == used and used and table[b, used - 1] >= 0 and b:
            lens[b] = max(0, min(used * page, int(rng.integers((used - 1) * page, used * page + 1))))
        if rng.random() < spare and used < width and free:
            table[b, used] = free.pop()
        if rng.random() < 0.1:
            table[b, width - 1] = table[b, width - 1] if table[b, width - 1] >= 0 else pages + int(rng.integers(5))
    refs = np.bincount(table[(table >= 0) & (table < pages)], minlength=pages).astype(np.int32)
    refs[rng.random(pages) < pins] += 1
    return table, lens, refs


SIZES = [(1, 1, 1, 16), (1, 4, 9, 16), (7, 5, 40, 16), (64, 20, 700, 32), (3, 300, 800, 64), (200, 3, 2500, 1024),
         (1500, 2, 4000, 16), (5, 70, 1024, 16), (16, 9, 1025, 128)]


@pytest.mark.parametrize("rows,width,pages,page", SIZES)
@pytest.mark.parametrize("seed", [1, 2])
def test_fork(rows, width, pages, page, seed):
    dev = device()
    log(f"fork {rows}x{width} of {pages}")
    rng = np.random.default_rng(seed)
    table, lens, refs = pool(rows, width, pages, page, rng)
    same = np.arange(rows)
    for parent in (same, same[::-1], rng.integers(-1, rows, rows), np.full(rows, -1), rng.integers(0, rows, 2 * rows + 3),
                   same[:rows // 2], rng.integers(-5, rows + 5, rows), np.zeros(rows, int)):
        parent = parent.astype(np.int32)
        args = [put(table, dev), put(lens, dev), put(refs, dev)]
        got = host(w4.kv_fork(*args, put(parent, dev), page))
        for a, b in zip(got, ref.fork(table, lens, refs, parent.tolist(), page)):
            assert a.shape == b.shape and (a == b).all()
        for a, b in zip(host(args), (table, lens, refs)):
            assert (a == b).all()                           # the arguments stay as they are


def check_alloc(table, lens, refs, tokens, page, dev, strided=False):
    tokens_each = np.zeros_like(lens) + np.asarray(tokens, np.int32)
    t = put(table, dev)
    if strided:
        wide = put(np.concatenate([table, np.full((len(table), 3), 5, np.int32)], axis=1), dev)
        t = wide[:, :table.shape[1]]
    arg = put(tokens_each, dev) if np.ndim(tokens) else int(tokens)
    got = host(w4.kv_alloc(t, put(lens, dev), put(refs, dev), arg, page))
    want = ref.alloc(table, lens, refs, [int(x) for x in tokens_each], page)
    for a, b in zip(got[:3], want[:3]):
        assert (a == b).all()
    pairs, missing = want[3], want[4]
    assert got[5].tolist() == [len(pairs), missing]
    assert list(zip(got[3].tolist(), got[4].tolist()))[:len(pairs)] == pairs
    assert (got[3][len(pairs):] == -1).all() and (got[4][len(pairs):] == -1).all()
    return want


@pytest.mark.parametrize("rows,width,pages,page", SIZES)
@pytest.mark.parametrize("seed", [3, 4])
def test_alloc(rows, width, pages, page, seed):
    """One token, none, many, each row its own number; pools that run out."""
    dev = device()
    log(f"alloc {rows}x{width} of {pages}")
    rng = np.random.default_rng(seed)
    table, lens, refs = pool(rows, width, pages, page, rng)
    check_alloc(table, lens, refs, 1, page, dev)
    check_alloc(table, lens, refs, 0, page, dev)
    check_alloc(table, lens, refs, 3 * page, page, dev, strided=True)
    check_alloc(table, lens, refs, rng.integers(-1, 2 * page, rows).astype(np.int32), page, dev)
    # after a fork, where rows share the pages that they go on writing
    parent = rng.integers(0, rows, rows).tolist()
    table, lens, refs = ref.fork(table, lens, refs, parent, page)
    check_alloc(table, lens, refs, 1, page, dev)
    check_alloc(table, lens, refs, rng.integers(0, 3, rows).astype(np.int32), page, dev)
    # nothing free, and nothing else in use
    check_alloc(table, lens, np.maximum(refs, 1), page, page, dev)
    check_alloc(np.full_like(table, -1), np.zeros_like(lens), np.zeros_like(refs), 2 * page + 1, page, dev)


def test_alloc_shared_pages():
    """Of the rows that write a shared page all but the last copy it; all of
    them where the page is held elsewhere too, or by a row that does not write."""
    dev = device()
    log("alloc shared")
    table = np.array([[0, 1, -1], [0, 1, -1], [0, 1, -1], [0, 2, -1]], np.int32)
    lens = np.array([20, 20, 20, 32], np.int32)
    refs = np.array([4, 3, 1, 0, 0, 0, 0, 0], np.int32)
    want = check_alloc(table, lens, refs, 1, 16, dev)
    assert want[3] == [(1, 3), (1, 4)] and want[0][2, 1] == 1 and want[0][3, 2] == 5
    want = check_alloc(table, lens, refs, np.array([1, 0, 1, 0], np.int32), 16, dev)
    assert want[3] == [(1, 3), (1, 4)]                     # row 1 keeps it
    refs[1] = 4
    assert len(check_alloc(table, lens, refs, 1, 16, dev)[3]) == 3
    # one free page for two copies: the second row is left without
    refs = np.array([4, 4, 1, 0, 1, 1, 1, 1], np.int32)
    want = check_alloc(table[:2], lens[:2], refs, 1, 16, dev)
    assert want[3] == [(1, 3)] and want[4] == 1 and want[0][1, 1] == -1


@pytest.mark.parametrize("rows,width,pages,page", SIZES)
@pytest.mark.parametrize("live", [0.0, 0.3, 1.0])
def test_compact(rows, width, pages, page, live):
    dev = device()
    log(f"compact {rows}x{width} of {pages} live={live}")
    rng = np.random.default_rng(5)
    table, _, refs = pool(rows, width, pages, page, rng, pins=live)
    if live == 0.0 and rows > 5:
        table[:], refs[:] = -1, 0
        refs[0] = -3
    args = [put(table, dev), put(refs, dev)]
    got = host(w4.kv_compact(*args))
    want = ref.compact(table, refs)
    for a, b in zip(got[:3], want[:3]):
        assert (a == b).all()
    pairs = want[3]
    assert got[5].tolist() == [len(pairs), 0]
    assert list(zip(got[3].tolist(), got[4].tolist()))[:len(pairs)] == pairs
    assert (got[3][:pages // 2][len(pairs):] == -1).all()
    assert (host(args)[0] == table).all() and (host(args)[1] == refs).all()


def test_large_pool():
    """More blocks of pages than a workgroup has threads."""
    dev = device()
    log("pages large pool")
    rng = np.random.default_rng(6)
    pages = (1 << 20) + 1030
    refs = (rng.random(pages) < 0.6).astype(np.int32)
    refs[:900000] = 1
    table = rng.integers(900000, pages, (20, 50)).astype(np.int32)
    refs[table] = 2
    got = host(w4.kv_compact(put(table, dev), put(refs, dev)))
    want = ref.compact(table, refs)
    for a, b in zip(got[:3], want[:3]):
        assert (a == b).all()
    table[:, 20:] = -1
    check_alloc(table, np.full(20, 20 * 16, np.int32), refs, 400, 16, dev)


@pytest.mark.parametrize("heads,page,dim", [(1, 16, 16), (8, 64, 128), (3, 32, 80), (2, 1024, 256)])
def test_copy_pages(heads, page, dim):
    """Pairs that name no page, counts below and beyond, one pair and many, and
    a cache whose pages have strides of their own."""
    import torch
    dev = device()
    log(f"copy pages {heads}x{page}x{dim}")
    rng = np.random.default_rng(7)
    for layers in (1, 2):
        cache = put(rng.integers(-127, 128, (40, layers, 2, heads, page, dim)).astype(np.int8), dev)
        scale = put(rng.random((40, layers, 2, heads)).astype(np.float16), dev)
        src, dst = rng.permutation(40).astype(np.int32)[:30].reshape(2, 15)
        src, dst = src.copy(), dst.copy()
        src[3], dst[5], src[9], dst[10] = -1, 40, 1 << 30, -7
        for count in (None, 0, 1, 7, 15, 1000, -2):
            c, s = cache.clone(), scale.clone()
            w4.kv_copy_pages(c[:, 0], s[:, 0], put(src, dev), put(dst, dev),
                             None if count is None else put(np.array([count, 9], np.int32), dev))
            torch.cuda.synchronize()
            want_c, want_s = cache.clone(), scale.clone()
            for i in range(15 if count is None else max(0, min(count, 15))):
                if 0 <= src[i] < 40 and 0 <= dst[i] < 40:
                    want_c[int(dst[i]), 0] = cache[int(src[i]), 0]
                    want_s[int(dst[i]), 0] = scale[int(src[i]), 0]
            assert torch.equal(c, want_c) and torch.equal(s, want_s)
    w4.kv_copy_pages(cache[:, 0], scale[:, 0], put(src[:0], dev), put(dst[:0], dev))


def test_copy_far_pages():
    import torch
    dev = device()
    log("copy far pages")
    far = torch.zeros(4 * (3 << 29) + 4096, dtype=torch.int8, device=dev)
    cache = far.as_strided((4, 2, 2, 16, 64), (3 << 29, 2048, 1024, 64, 1))
    scale = torch.rand((4, 2, 2), device=dev).half()
    cache[0] = torch.arange(4096, device=dev).view(2, 2, 16, 64).to(torch.int8)
    w4.kv_copy_pages(cache, scale, put(np.array([0], np.int32), dev), put(np.array([3], np.int32), dev))
    torch.cuda.synchronize()
    assert torch.equal(cache[3], cache[0]) and torch.equal(scale[3], scale[0]) and not cache[1:3].any()


def test_captured_beam_step():
    """Fork, alloc and copy in one graph; each replay equals the eager step."""
    import torch
    dev = device()
    log("captured beam step")
    rng = np.random.default_rng(8)
    rows, width, pages, page = 24, 8, 400, 16
    states = [pool(rows, width, pages, page, rng) for _ in range(4)]
    parents = [rng.integers(0, rows, rows).astype(np.int32) for _ in states]
    codes = rng.integers(-127, 128, (pages, 2, 2, page, 32)).astype(np.int8)
    scales = rng.random((pages, 2, 2)).astype(np.float16)
    table, lens, refs = (put(a, dev) for a in states[0])
    parent, cache, scale = put(parents[0], dev), put(codes, dev), put(scales, dev)

    def step():
        t, l, r = w4.kv_fork(table, lens, refs, parent, page)
        t, l, r, src, dst, counts = w4.kv_alloc(t, l, r, 1, page)
        w4.kv_copy_pages(cache, scale, src, dst, counts)
        return t, l, r, src, dst, counts

    def fill(i):
        for t, a in zip((table, lens, refs, parent, cache, scale), (*states[i], parents[i], codes, scales)):
            t.copy_(put(a, dev))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        fill(i)
        eager = [t.clone() for t in step()] + [cache.clone(), scale.clone()]
        fill(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, [*out, cache, scale]):
            assert torch.equal(a, b)
        t, l, r = ref.fork(*states[i], parents[i].tolist(), page)
        assert (eager[0].cpu().numpy() == ref.alloc(t, l, r, [1] * rows, page)[0]).all()
        (torch.rand(1000, device=dev) * 2).sum().item()
