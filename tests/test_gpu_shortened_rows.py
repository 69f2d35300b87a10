"""Whose pages are written: after kv_alloc every page that a row's new tokens
reach is named by nobody else, also for rows that were forked and then shortened,
once they have given up the pages behind their tokens."""
import numpy as np
import pytest

import w4a8_gemm_amd as w4
from gpu_util import device, log

pytestmark = pytest.mark.gpu


def put(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def give_up(table, lens, refs, page):
    """The rows without the pages behind their tokens: continued in other rows."""
    import torch
    rows = table.shape[0]
    parent = torch.arange(2 * rows, dtype=torch.int32, device=table.device) - rows       # < 0: none
    table, lens, refs = w4.kv_fork(table, lens, refs, parent, page)
    return table[rows:], lens[rows:], refs


def check_written(table, before, lens, refs, page):
    """Every entry that new tokens reach has a page of its own, or of writers
    before whom all others have left it."""
    table, before, lens, refs = (t.cpu().numpy() for t in (table, before, lens, refs))
    named = np.bincount(table[table >= 0], minlength=len(refs))
    assert (named <= refs).all()
    for row, lo, hi in zip(table, before, lens):
        for column in range(lo // page, -(-hi // page) if hi > lo else 0):
            assert row[column] >= 0 and refs[row[column]] == 1


@pytest.mark.parametrize("back", [39, 33, 32, 31, 16, 10, 0])
@pytest.mark.parametrize("pinned", [False, True])
def test_a_forked_row_taken_back(back, pinned):
    """A and B share 40 tokens, B is taken back and goes on: what A sees stays, and
    what something else holds."""
    import torch
    dev = device()
    log(f"taken back to {back} pinned={pinned}")
    rng = np.random.default_rng(back)
    cache = put(rng.integers(-127, 128, (12, 2, 2, 16, 64)).astype(np.int8), dev)
    scale = put((rng.random((12, 2, 2)) / 127).astype(np.float16), dev)
    table = put(np.array([[7, 3, 5, -1], [-1, -1, -1, -1]], np.int32), dev)
    refs = torch.zeros(12, dtype=torch.int32, device=dev)
    refs[[3, 5, 7]] = 1 + int(pinned)
    lens = put(np.array([40, 0], np.int32), dev)
    table, lens, refs = w4.kv_fork(table, lens, refs, put(np.zeros(2, np.int32), dev), 16)
    assert refs[[3, 5, 7]].tolist() == [2 + int(pinned)] * 3
    lens[1] = back
    table, lens, refs = give_up(table, lens, refs, 16)
    kept = -(-back // 16)
    assert (table[1, kept:] == -1).all() and torch.equal(table[1, :kept], table[0, :kept])
    before = lens.clone()
    table, lens, refs, src, dst, counts = w4.kv_alloc(table, lens, refs, 20, 16)
    w4.kv_copy_pages(cache, scale, src, dst, counts)
    torch.cuda.synchronize()
    assert counts[1] == 0
    check_written(table, before, lens, refs, 16)
    codes, scales = cache.clone(), scale.clone()
    k = put(8 * rng.standard_normal((40, 2, 64)).astype(np.float16), dev)
    w4.rope_append(k, k, k, None, cache, scale, table[1:], lens[1:], cu_q=put(np.array([0, 20], np.int32), dev))
    torch.cuda.synchronize()
    theirs = torch.ones(12, dtype=torch.bool, device=dev)
    theirs[table[1, back // 16:-(-(back + 20) // 16)].long()] = False
    assert theirs[table[0, :4].long()].all() and (not pinned or theirs[[3, 5, 7]].all())
    assert torch.equal(cache[theirs], codes[theirs]) and torch.equal(scale[theirs], scales[theirs])


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("seed", range(4))
def test_many_steps(seed, page):
    """Steps that allocate, confirm some of the tokens, fork, now and then shorten
    rows by any number, and compact."""
    import torch
    dev = device()
    log(f"many steps seed={seed} page={page}")
    rng = np.random.default_rng(seed)
    rows, width, pages = 12, 9, 150
    table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(rows, dtype=torch.int32, device=dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    written = 0
    for step in range(40):
        room = width * page - lens.cpu().numpy()
        tokens = np.minimum(rng.integers(0, 2 * page + 1, rows), room).astype(np.int32)
        before = lens
        table, lens, refs, _, _, counts = w4.kv_alloc(table, lens, refs, put(tokens, dev), page)
        assert counts[1] == 0
        check_written(table, before, lens, refs, page)
        written += int(tokens.sum())
        # confirmed: as many tokens as tree_accept may, one at least
        lens = before + put(np.minimum(tokens, rng.integers(1, 2 * page + 1, rows)).astype(np.int32), dev)
        named = torch.bincount(table[table >= 0], minlength=pages).int()
        assert torch.equal(named, refs)
        kind = step % 4
        if kind == 1:
            table, lens, refs = w4.kv_fork(table, lens, refs, put(rng.integers(-1, rows, rows).astype(np.int32), dev), page)
        elif kind == 2:
            lens = put(rng.integers(0, lens.cpu().numpy() + 1).astype(np.int32), dev)
            table, lens, refs = give_up(table, lens, refs, page)
        elif kind == 3:
            table, refs = w4.kv_compact(table, refs)[:2]
    assert written > 1000
