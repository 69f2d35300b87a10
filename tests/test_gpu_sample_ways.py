"""sample() on both sides of the sizes where it goes another way: rows that are
looked at by several workgroups before, and counts that the largest logits of
128-byte groups bound."""
import numpy as np
import pytest

import w4a8_gemm_amd as w4
from gpu_util import device, log
from test_gpu_sample import FILTERS, check, logits, put, run

pytestmark = pytest.mark.gpu

LONG_ROW = 24576


def test_the_row_length_that_these_tests_are_about():
    for f32 in (0, 1):
        assert w4.lib.w4a8_sample_workspace_size(f32, 5, LONG_ROW - 1) == 0
        assert w4.lib.w4a8_sample_workspace_size(f32, 5, LONG_ROW) > 0


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("vocab", [LONG_ROW - 1, LONG_ROW, LONG_ROW + 1])
def test_shortest_long_rows(vocab, dtype):
    """Flat, steep, tied, nearly empty and ordinary rows that begin at any place,
    with every kind of filter and with settings of each row."""
    dev = device()
    log(f"sample ways vocab={vocab} {dtype.__name__}")
    rng = np.random.default_rng(vocab)
    wide = np.full((9, vocab + 5), 60000, dtype)
    x = wide[:, 3:3 + vocab]
    x[:] = logits(9, vocab, rng, dtype)
    x[0] = (0.01 * rng.standard_normal(vocab)).astype(dtype)
    x[1] = (30 * rng.standard_normal(vocab)).astype(dtype)
    x[2] = rng.integers(0, 3, vocab)
    x[3] = -np.inf
    x[3, [0, vocab - 1]] = 1.0
    x[4] = 1.0
    x[5, vocab - 1] = np.nan
    u = rng.random(9).astype(np.float32)
    part = put(wide, dev)[:, 3:3 + vocab]
    for filters in FILTERS + [dict(top_k=vocab - 1, top_p=0.9), dict(min_p=1e-4), dict(min_p=0.5, top_p=0.99)]:
        check(x, u, *run(part, u, dev, **filters), **filters)
    each = dict(top_k=rng.choice([0, 5, 700], 9).astype(np.int32), top_p=rng.choice([0.7, 1.0], 9).astype(np.float32),
                temperature=rng.choice([0.0, 1.0], 9).astype(np.float32), min_p=rng.choice([0.0, 0.1], 9).astype(np.float32))
    check(x, u, *run(part, u, dev, **each), **each)


@pytest.mark.parametrize("dtype,each", [(np.float16, 64), (np.float32, 32)])
def test_counts_around_the_number_of_groups(dtype, each):
    """More tokens asked for than there are groups: no bound comes from their
    largest; up to twice as many as a list holds, all of them finite or few."""
    dev = device()
    log(f"sample ways counts {dtype.__name__}")
    rng = np.random.default_rng(each)
    vocab = 32000
    x, u = logits(5, vocab, rng, dtype), rng.random(5).astype(np.float32)
    x[1, 300:] = -np.inf
    x[2] = rng.integers(0, 4, vocab)
    groups = vocab // each
    for top_k in (groups - 1, groups, groups + 1, groups + 2, 2047, 2048, 2049, 8192):
        for top_p in (1.0, 0.8):
            check(x, u, *run(x, u, dev, top_k=top_k, top_p=top_p), top_k=top_k, top_p=top_p)
