"""Sizes, strides and bounds beyond the C interface's int (no GPU): fake CUDA
tensors and a stand-in for the library that keeps what it was passed."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import w4a8_gemm_amd as w4

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")

BIG = 2 ** 32          # its low 32 bits are 0


@pytest.fixture
def calls(monkeypatch):
    log = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *args: 0
            return lambda *args: log.append(args) or 0

    with FakeTensorMode():
        monkeypatch.setattr(w4, "lib", Lib())
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x10)
        yield log


def fake(shape, stride, dtype=torch.float16):
    return torch.empty_strided(shape, stride, dtype=dtype, device="cuda:0")


def state(table_ld=8, batch=2, **kw):
    return (fake((9, 2, 2, 16, 64), (4096, 2048, 1024, 64, 1), torch.int8), fake((9, 2, 2), (4, 2, 1)),
            fake((batch, 8), (table_ld, 1), torch.int32), fake((batch,), (1,), torch.int32))


def test_strides_and_sizes_are_refused(calls):
    x, wide, w = fake((2, 64), (64, 1)), fake((2, 64), (BIG + 64, 1)), fake((64,), (1,))
    i8 = fake((2, 64), (BIG + 64, 1), torch.int8)
    q, k = fake((2, 4, 64), (256, 64, 1)), fake((2, 2, 64), (128, 64, 1))
    q_far, k_far = fake((2, 4, 64), (BIG + 256, 64, 1)), fake((2, 2, 64), (BIG + 128, 64, 1))
    for bad in (lambda: w4.rms_norm_quant(wide, w), lambda: w4.rms_norm_quant(x, w, residual=wide),
                lambda: w4.rms_norm_quant(x, w, h=wide), lambda: w4.rms_norm_quant(x, w, a8=i8),
                lambda: w4.silu_mul_quant(wide), lambda: w4.silu_mul_quant(x, wide),
                lambda: w4.silu_mul_quant(x, x, a8=i8), lambda: w4.silu_mul_quant(fake((BIG + 2, 2), (2, 1))),
                lambda: w4.silu_mul_quant(fake((1, BIG + 64), (BIG + 64, 1))),
                lambda: w4.rope_append(q_far, k, k, None, *state()),
                lambda: w4.rope_append(q, k_far, k, None, *state()),
                lambda: w4.rope_append(q, k, k_far, None, *state()),
                lambda: w4.rope_append(q, k, k, None, *state(), out=q_far),
                lambda: w4.rope_append(q, k, k, fake((BIG + 8, 64), (64, 1), torch.float32), *state()),
                lambda: w4.rope_append(q, k, k, None, *state(BIG + 8)),
                lambda: w4.paged_attention(q_far, *state()),
                lambda: w4.paged_attention(q, *state(), out=q_far),
                lambda: w4.paged_attention(q, *state(BIG + 8))):
        with pytest.raises(ValueError):
            bad()
    assert not calls
    # the largest that fit go through
    w4.rms_norm_quant(fake((2, 64), (2 ** 31 - 1, 1)), w)
    w4.rope_append(fake((2, 4, 64), (2 ** 31 - 8, 64, 1)), k, k, None, *state(2 ** 31 - 1))
    assert len(calls) == 2


def test_bounds_and_windows_beyond_any_sequence(calls):
    q = fake((2, 4, 64), (256, 64, 1))
    w4.paged_attention(q, *state(), max_q=BIG + 1, max_len=BIG + 5, window=BIG + 5)
    assert (calls[0][4], calls[0][5], calls[0][7]) == (2 ** 31 - 1,) * 3     # max_q, max_len, window
