"""Where a call with stream= allocates and launches (no GPU): fake CUDA tensors,
a recording stand-in for the library and for torch's streams."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import w4a8_gemm_amd as w4

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")

M, N, K, G = 5, 256, 512, 128


def tensors(device="cuda:0"):
    half = lambda *shape: torch.empty(shape, dtype=torch.float16, device=device)
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)
    i8 = lambda *shape: torch.empty(shape, dtype=torch.int8, device=device)
    return types.SimpleNamespace(
        a=half(M, K), a8=i8(M, K), s_a=half(M), blob=i8(N * K).view(torch.uint8), weight=half(K),
        q=half(3, 4, 64), k=half(3, 2, 64), y=half(M, N), sink=i32(64),
        kv=(i8(9, 2, 2, 16, 64), half(9, 2, 2), i32(3, 8), i32(3)))


# name -> (call, buffers it allocates, tensors it returns)
CALLS = {
    "quant_act": (lambda t, **kw: w4.quant_act(t.a, **kw), 2, 2),
    "quant_act_static": (lambda t, **kw: w4.quant_act_static(t.a, 0.5, **kw), 2, 2),
    "gemm": (lambda t, **kw: w4.gemm(t.a8, t.s_a, t.blob, N, K, G, want_acc=True, **kw), 3, 2),
    "gemm_noalloc": (lambda t, **kw: w4.gemm_noalloc(t.a8, t.s_a, t.blob, N, K, G, t.y, **kw), 0, 0),
    "linear": (lambda t, **kw: w4.linear(t.a, t.blob, N, K, G, want_acc=True, **kw), 5, 4),
    "w4a16": (lambda t, **kw: w4.w4a16(t.a, t.blob, N, K, G, **kw), 1, 1),
    "rms_norm_quant": (lambda t, **kw: w4.rms_norm_quant(t.a, t.weight, residual=t.a, **kw), 3, 3),
    "rms_norm_quant, no residual": (lambda t, **kw: w4.rms_norm_quant(t.a, t.weight, **kw), 2, 2),
    "silu_mul_quant": (lambda t, **kw: w4.silu_mul_quant(t.a, **kw), 2, 2),
    "rope_append": (lambda t, **kw: w4.rope_append(t.q, t.k, t.k, None, *t.kv, **kw), 1, 1),
    "rope_append, in place": (lambda t, **kw: w4.rope_append(t.q, t.k, t.k, None, *t.kv, out=t.q, **kw), 0, 0),
    "paged_attention": (lambda t, **kw: w4.paged_attention(t.q, *t.kv, **kw), 2, 1),
    "read_probe": (lambda t, **kw: w4.read_probe(t.blob, 0, 4096, 4, t.sink, **kw), 0, 0),
}


class Stream:
    def __init__(self, handle, index=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


@pytest.fixture
def seen(monkeypatch):
    """Records (event, handle of the stream that was current)."""
    log = types.SimpleNamespace(empty=[], launched=[], recorded=[], caller=Stream(0x10))
    current = [log.caller]

    @contextlib.contextmanager
    def enter(stream):
        current.append(stream)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *args: 4096
            def launch(*args):
                log.launched.append(args[-1])
                return 0
            return launch

    empty = torch.empty
    mode = FakeTensorMode()
    with mode:
        log.tensors = tensors()

        def recorded_empty(*args, **kw):
            log.empty.append(current[-1].cuda_stream)
            return empty(*args, **kw)
        monkeypatch.setattr(w4, "lib", Lib())
        monkeypatch.setattr(torch, "empty", recorded_empty)
        monkeypatch.setattr(torch.cuda, "stream", enter)
        monkeypatch.setattr(torch.cuda, "set_stream", lambda stream: current.__setitem__(-1, stream))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: current[-1].cuda_stream)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, stream: log.recorded.append((id(t), stream.cuda_stream)))
        yield log


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_stream_they_are_used_on(seen, name):
    call, allocated, returned = CALLS[name]
    out = call(seen.tensors, stream=Stream(0x20))
    assert seen.launched == [0x20]
    assert seen.empty == [0x20] * allocated
    # new results are read on the caller's stream: freeing one waits for that too
    out = out if isinstance(out, tuple) else (out,)
    assert len(seen.recorded) == returned and all(s == 0x10 for _, s in seen.recorded)
    assert {i for i, _ in seen.recorded} <= {id(t) for t in out}


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_by_default(seen, name):
    call, allocated, _ = CALLS[name]
    call(seen.tensors)
    assert seen.launched == [0x10] and seen.empty == [0x10] * allocated and not seen.recorded
