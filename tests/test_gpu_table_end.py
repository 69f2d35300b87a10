"""Sequences that run past the end of their row of the block table: what lies
there is not written, and what lies before stays as it is, so that a step for
which the table had no room can be taken back."""
import numpy as np
import pytest

import w4a8_gemm_amd as w4
from gpu_util import device, log
from test_gpu_kv_cache import Batch, check_append

pytestmark = pytest.mark.gpu


def put(a, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def cut(batch, dev, entries):
    """The batch's device state with only the first entries of the block table."""
    st = batch.device(dev)
    st["block_table"] = st["block_table"][:, :entries]
    return st


def append(batch, st, qkv, heads, cos_sin):
    import torch
    q, k, v = qkv.split([heads, batch.kv_heads, batch.kv_heads], dim=1)
    q = w4.rope_append(q, k, v, cos_sin, st["cache"], st["scale"], st["block_table"], st["seq_lens"], cu_q=st["cu_q"])
    torch.cuda.synchronize()
    return q.cpu().numpy(), st["cache"].cpu().numpy(), st["scale"].cpu().numpy()


# (length with the new tokens, new tokens); the table holds 32 positions
ENDS = [(33, 1), (36, 8), (32, 3), (64, 32), (40, 0), (70, 70), (20, 4), (45, 1)]


@pytest.mark.parametrize("page,entries", [(16, 2), (32, 1)])
@pytest.mark.parametrize("kv_heads,dim", [(2, 64), (1, 128), (3, 16)])
@pytest.mark.parametrize("spans", [ENDS, [(33, 1), (32, 1), (5, 1), (64, 1)]])
def test_append(page, entries, kv_heads, dim, spans):
    """As with a table whose entries from there on name no page."""
    dev = device()
    log(f"append past the table page={page} heads={kv_heads} dim={dim} {len(spans)} sequences")
    batch = Batch(spans, page, kv_heads, dim, 1, cu=spans is ENDS)
    batch.table[:, entries:] = -1
    qkv = batch.rng.standard_normal((batch.tokens, 2 + 2 * kv_heads, dim)).astype(np.float16)
    angles = w4.rope_table(60, dim, device=dev)
    wide = append(batch, batch.device(dev), put(qkv, dev), 2, angles)
    check_append(batch, qkv, 2, angles.cpu().numpy(), False, *wide)
    narrow = append(batch, cut(batch, dev, entries), put(qkv, dev), 2, angles)
    for a, b in zip(wide, narrow):
        assert (a.view(np.uint8) == b.view(np.uint8)).all()


def test_append_at_the_largest_lengths():
    """Lengths up to 2^31 - 1 write nothing; what has negative ones is no worse."""
    dev = device()
    log("append largest lengths")
    batch = Batch([(32, 4), (32, 2), (32, 1), (32, 5)], 16, 2, 64, 2)
    batch.lens[:] = 2 ** 31 - 1, 2 ** 31 - 1024, 2 ** 31 - 16, 37
    qkv = batch.rng.standard_normal((batch.tokens, 6, 64)).astype(np.float16)
    _, cache, scale = append(batch, batch.device(dev), put(qkv, dev), 2, None)
    assert (cache == batch.cache).all() and (scale == batch.scale).all()


def test_a_step_without_room_is_taken_back():
    """Two answers share full pages up to the table's end.  The step that one
    more token each would need finds no room; the old table, lengths and counts
    are the cache before it."""
    import torch
    dev = device()
    log("no room, taken back")
    rng = np.random.default_rng(3)
    cache = put(rng.integers(-127, 128, (6, 2, 2, 16, 64)).astype(np.int8), dev)
    scale = put((rng.random((6, 2, 2)) / 127).astype(np.float16), dev)
    table = put(np.array([[4, 1], [4, 1], [0, -1]], np.int32), dev)
    lens = put(np.array([32, 32, 9], np.int32), dev)
    refs = put(np.array([1, 2, 0, 0, 2, 0], np.int32), dev)
    before, scales = cache.clone(), scale.clone()
    new_table, new_lens, _, src, dst, counts = w4.kv_alloc(table, lens, refs, 3, 16)
    w4.kv_copy_pages(cache, scale, src, dst, counts)
    q = put(rng.standard_normal((9, 4, 64)).astype(np.float16), dev)
    k = put(8 * rng.standard_normal((9, 2, 64)).astype(np.float16), dev)
    cu = put(np.array([0, 3, 6, 9], np.int32), dev)
    w4.rope_append(q, k, k, None, cache, scale, new_table, new_lens, cu_q=cu)
    path = put(np.tile(np.array([0, 2], np.int32), (3, 1)), dev)
    w4.kv_keep(cache, scale, new_table, new_lens, path, put(np.full(3, 2, np.int32), dev), cu_q=cu)
    torch.cuda.synchronize()
    assert counts.tolist() == [0, 2] and new_lens.tolist() == [35, 35, 12]
    assert torch.equal(cache[[1, 4]], before[[1, 4]]) and torch.equal(scale[[1, 4]], scales[[1, 4]])
    assert not torch.equal(cache[0], before[0])                     # the third one had room


@pytest.mark.parametrize("page,entries", [(16, 2), (32, 1)])
def test_keep(page, entries):
    """Confirmed nodes past the table's end are not there, places there not
    written: as with a table whose entries from there on name no page."""
    import torch
    dev = device()
    log(f"keep past the table page={page}")
    spans = [(36, 8), (33, 1), (50, 20), (40, 30), (64, 16), (32, 6), (70, 70)]
    batch = Batch(spans, page, 2, 64, 4)
    batch.table[:, entries:] = -1
    path = np.full((len(spans), 9), -1, np.int32)
    count = np.zeros(len(spans), np.int32)
    for b, (_, n) in enumerate(spans):
        line = [0] + sorted(batch.rng.choice(np.arange(1, n), min(n - 1, 8), replace=False).tolist())
        path[b, :len(line)], count[b] = line, len(line)
    outs = []
    for st in (batch.device(dev), cut(batch, dev, entries)):
        w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], put(path, dev), put(count, dev),
                   cu_q=st["cu_q"])
        torch.cuda.synchronize()
        outs.append(st)
    assert torch.equal(outs[0]["cache"], outs[1]["cache"]) and torch.equal(outs[0]["scale"], outs[1]["scale"])
    assert (outs[0]["cache"].cpu().numpy() != batch.cache).any()
    batch.lens[:] = 2 ** 31 - 1
    st = batch.device(dev)
    w4.kv_keep(st["cache"], st["scale"], st["block_table"], st["seq_lens"], put(path, dev), put(count, dev),
               cu_q=st["cu_q"])
    torch.cuda.synchronize()
    assert (st["cache"].cpu().numpy() == batch.cache).all()
