"""kv_alloc's count of entries without a page where it is large."""
import numpy as np
import pytest

import w4a8_gemm_amd as w4
from gpu_util import device, log

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width,page", [(1, 3, 16), (15, 1, 16), (17, 2, 16), (32, 3, 16), (2000, 2, 16), (33, 1, 1024)])
@pytest.mark.parametrize("tokens", [2 ** 31 - 1, 2 ** 30, 100000])
def test_entries_beyond_the_table(rows, width, page, tokens):
    """Every entry that the new tokens reach counts, up to 2^31 - 1; 32 rows of
    2^31 - 1 tokens in pages of 16 reach 2^32."""
    import torch
    dev = device()
    log(f"alloc counts {rows}x{width} page={page} tokens={tokens}")
    table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    zeros = torch.zeros(rows, dtype=torch.int32, device=dev)
    for pages_free in (0, 1):
        refs = torch.tensor([1 - pages_free, 1], dtype=torch.int32, device=dev)
        for new in (tokens, zeros + tokens):
            out, lens, _, _, _, counts = w4.kv_alloc(table, zeros, refs, new, page)
            torch.cuda.synchronize()
            want = rows * -(-tokens // page) - pages_free
            assert counts.tolist() == [0, min(want, 2 ** 31 - 1)]
            assert (lens == tokens).all() and int((out >= 0).sum()) == pages_free
