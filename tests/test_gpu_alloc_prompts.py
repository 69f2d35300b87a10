"""kv_alloc for prompts: hundreds of pages a row, among pages that the row has
and pages that others hold."""
import numpy as np
import pytest

from gpu_util import device, log
from test_gpu_kv_pages import check_alloc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width,pages,page", [(1, 513, 600, 16), (6, 600, 4000, 16), (3, 130, 2100, 64), (70, 129, 9000, 32)])
@pytest.mark.parametrize("held", [0.0, 0.4])
def test_prompts(rows, width, pages, page, held):
    dev = device()
    log(f"alloc prompts {rows}x{width} of {pages} held={held}")
    rng = np.random.default_rng(rows)
    refs = (rng.random(pages) < held).astype(np.int32)
    table, lens = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32)
    whole = np.full(rows, width * page, np.int32)
    check_alloc(table, lens, refs, whole, page, dev)
    check_alloc(table, lens, refs, rng.integers(0, width * page + 200, rows).astype(np.int32), page, dev)
    # after some tokens, with pages here and there that the row has already
    free = np.flatnonzero(refs == 0)
    rng.shuffle(free)
    free = free.tolist()
    for b in range(rows):
        lens[b] = rng.integers(0, 3 * page)
        for c in range(width):
            if c * page < lens[b] or rng.random() < 0.1:
                if free:
                    table[b, c] = free.pop()
                    refs[table[b, c]] = 1
    check_alloc(table, lens, refs, whole, page, dev)
    check_alloc(table, lens, refs, rng.integers(0, width * page, rows).astype(np.int32), page, dev, strided=True)
    # none free from the middle of a row on
    refs[np.flatnonzero(refs == 0)[width // 2:]] = 1
    check_alloc(table, lens, refs, whole, page, dev)
