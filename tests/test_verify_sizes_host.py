"""Numbers beyond the C interface's int (no GPU): ctypes would pass their low 32
bits."""
import pytest
import torch

import w4a8_gemm_amd as w4
from test_int_range_host import BIG, calls, fake, state  # noqa: F401  (calls: a fixture)

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
i32 = torch.int32


def row(n):
    return fake((n,), (1,), i32)


def test_page_sizes(calls):
    _, _, table, lens = state()
    refs = row(9)
    for page in (BIG + 16, BIG, -BIG + 16, -16, 2 ** 31):
        for bad in (lambda: w4.kv_fork(table, lens, refs, row(2), page), lambda: w4.kv_alloc(table, lens, refs, 1, page),
                    lambda: w4.kv_alloc(table, lens, refs, row(2), page)):
            with pytest.raises(ValueError):
                bad()
    assert not calls
    w4.kv_fork(table, lens, refs, row(2), 16)
    w4.kv_alloc(table, lens, refs, 1, 16)
    assert calls[0][7] == calls[1][7] == 16


def test_lengths_of_tensors(calls):
    _, _, table, lens = state()
    cache, scale = state()[:2]
    nodes = row(BIG + 3)
    for bad in (lambda: w4.tree_mask(nodes, row(3), cu_q=row(4), max_q=7), lambda: w4.tree_mask(row(3), nodes, cu_q=row(BIG + 4)),
                lambda: w4.tree_accept(nodes, nodes, nodes, row(3), cu_q=row(4), max_q=7),
                lambda: w4.kv_fork(table, lens, row(9), nodes, 16), lambda: w4.kv_copy_pages(cache, scale, nodes, nodes)):
        with pytest.raises(ValueError):
            bad()
    assert not calls


@pytest.mark.parametrize("name", ["max_q", "max_len", "window"])
def test_bounds_below_the_range(calls, name):
    """They reach the library negative, which refuses them."""
    q = fake((2, 4, 64), (256, 64, 1))
    for value in (-1, -2 ** 31, -BIG, -BIG + 5, -2 ** 31 - 1):
        w4.paged_attention(q, *state(), **{name: value})
        w4.tree_attention(q, *state(), fake((2, 1), (1, 1), i32), **{name: value})
        for args, at in ((calls.pop(-2), (4, 5, 7)), (calls.pop(-1), (7, 8, 10))):
            passed = args[dict(zip(("max_q", "max_len", "window"), at))[name]]
            assert -2 ** 31 <= passed < 0


@pytest.mark.parametrize("pages", [1, 2, 9])
def test_pairs_of_a_compaction(calls, pages):
    """Half as many as pages, none of a single one: the kernels write no more."""
    _, _, src, dst, _ = w4.kv_compact(state()[2], row(pages))[1:]
    assert src.shape == dst.shape == (pages // 2,)
