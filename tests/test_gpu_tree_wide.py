"""tree_attention with 32 rows a workgroup, which the plan takes where there is
much work: every head dim's form, pages of 16 and more, windows, rows split over
their keys and not, against the same 64-bit numpy and bound as with 16."""
import ctypes

import numpy as np
import pytest

import w4a8_gemm_amd as w4
from gpu_util import device, log
from test_gpu_kv_cache import Batch
from test_gpu_tree import SPANS, attend, check, mask_of, put, trees

pytestmark = pytest.mark.gpu

MUCH = 1 << 22                # a bound on lengths for which there is much work
LONG = SPANS + [(2500, 40)]


def rows_of_a_workgroup(st, tokens, heads, max_q, max_len):
    """From the workspace's size, where rows are split: for each of about 512
    parts 16 or 32 rows of a maximum, a sum and dim values."""
    pages, _, kv_heads, page, dim = st["cache"].shape
    batch, entries = st["block_table"].shape
    v = w4.KvView(1024, 1024, 2 * kv_heads * page * dim, 2 * kv_heads, pages, page, kv_heads, dim, 1024, entries, entries,
                  1024, 1024, batch, tokens)
    size = w4.lib.w4a8_tree_attention_workspace_size(ctypes.byref(v), heads, max_q, max_len)
    return size // (512 // kv_heads * kv_heads * (8 + 4 * dim))


@pytest.mark.parametrize("window", [0, 1, 40, 1000])
@pytest.mark.parametrize("page,heads,kv_heads,dim", [
    (16, 4, 1, 64), (64, 4, 1, 64), (16, 3, 1, 16), (32, 6, 2, 48), (16, 8, 2, 128), (64, 8, 2, 128), (16, 6, 2, 80),
    (128, 5, 1, 96), (16, 3, 1, 256), (64, 4, 2, 256), (16, 2, 2, 192), (32, 4, 1, 192), (64, 32, 1, 128)])
def test_split_rows(page, heads, kv_heads, dim, window):
    dev = device()
    log(f"tree attention 32 rows page={page} heads={heads}/{kv_heads} dim={dim} window={window}")
    batch = Batch(LONG, page, kv_heads, dim, 31)
    parents, see = trees(batch, roots=True)
    q = (2 * batch.rng.standard_normal((batch.tokens, heads, dim))).astype(np.float16)
    st = batch.device(dev)
    mask, _ = w4.tree_mask(put(parents, dev), st["seq_lens"], cu_q=st["cu_q"], max_q=130)
    assert rows_of_a_workgroup(st, batch.tokens, heads, 130, 200) == 0
    assert rows_of_a_workgroup(st, batch.tokens, heads, 130, MUCH) == 32
    check(batch, q, see, attend(batch, q, mask, dev, window, state=st, max_q=130, max_len=MUCH), window)


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("page,dim", [(16, 64), (64, 64), (16, 32), (16, 128), (32, 80), (16, 256), (64, 256), (64, 208)])
def test_rows_that_are_not_split(page, dim, window):
    """As many row tiles as there may be workgroups: the 32-row tiles of 16 heads."""
    dev = device()
    log(f"tree attention 32 rows, not split page={page} dim={dim} window={window}")
    batch = Batch(SPANS, page, 16, dim, 32)
    _, see = trees(batch)
    q = (2 * batch.rng.standard_normal((batch.tokens, 32, dim))).astype(np.float16)
    st = batch.device(dev)
    assert batch.tokens * 2 // 32 + len(SPANS) >= 512 // 16
    assert rows_of_a_workgroup(st, batch.tokens, 32, 130, MUCH) == 0
    check(batch, q, see, attend(batch, q, mask_of(see, 5), dev, window, state=st, max_q=130, max_len=MUCH), window)


@pytest.mark.parametrize("page,dim", [(16, 128), (64, 256), (16, 80)])
def test_any_mask(page, dim):
    """Masks that are no trees, rows that see nothing, absent pages, a scale of 0,
    a NaN in a query."""
    dev = device()
    log(f"tree attention 32 rows, any mask page={page} dim={dim}")
    batch = Batch(LONG, page, 1, dim, 33)
    see = [batch.rng.random((n, n)) < batch.rng.choice([0.05, 0.5, 0.95], (n, 1)) for _, n in batch.spans]
    see[0][:] &= np.arange(70)[:, None] % 3 > 0
    batch.table[2, 1] = -1
    batch.table[7, 0] = batch.pages + 1
    batch.scale[batch.table[9, 1], 1] = 0
    q = (2 * batch.rng.standard_normal((batch.tokens, 4, dim))).astype(np.float16)
    q[80, 1, 3] = np.nan
    for window in (0, 25):
        o = attend(batch, q, mask_of(see, 5), dev, window, max_q=130, max_len=MUCH)
        clean = q.copy()
        clean[80, 1] = 0
        assert np.isnan(o[80, 1]).all()
        o[80, 1] = attend(batch, clean, mask_of(see, 5), dev, window, max_q=130, max_len=MUCH)[80, 1]
        check(batch, clean, see, o, window)
        assert (o[:70][::3] == 0).all()


def test_tables_so_wide_that_work_is_counted_coarsely():
    """A block table for 2^30 keys a sequence, of which few are there."""
    import torch
    dev = device()
    log("tree attention widest table")
    batch = Batch([(3000, 40), (70, 33), (1, 1), (0, 0)], 1024, 2, 64, 34)
    _, see = trees(batch)
    q = (2 * batch.rng.standard_normal((batch.tokens, 8, 64))).astype(np.float16)
    st = batch.device(dev)
    wide = torch.full((4, 1 << 20), -1, dtype=torch.int32, device=dev)
    wide[:, :batch.table.shape[1]] = st["block_table"]
    st["block_table"] = wide
    for most, length in ((40, None), (1, 1000), (40, 3000)):
        check(batch, q, see, attend(batch, q, mask_of(see, 2), dev, state=st, max_q=most, max_len=length))
