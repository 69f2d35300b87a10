"""Calls on tensors of a device that is not current, and on tensors of several
devices (no GPU): fake CUDA tensors and a stand-in for the library."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import w4a8_gemm_amd as w4
from test_streams_host import CALLS, K, M, Stream, tensors

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")


@pytest.fixture
def seen(monkeypatch):
    """Records the device that is current at each launch."""
    log = types.SimpleNamespace(launched=[])
    current = [0]

    @contextlib.contextmanager
    def enter(index):
        current.append(torch.device("cuda", index).index if isinstance(index, int) else index.index)
        yield
        current.pop()

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace_size"):
                return lambda *args: 4096
            return lambda *args: log.launched.append(current[-1]) or 0

    with FakeTensorMode():
        monkeypatch.setattr(w4, "lib", Lib())
        monkeypatch.setattr(torch.cuda, "device", enter)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(0x10, current[-1]))
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0x10)
        yield log


@pytest.mark.parametrize("name", CALLS)
def test_launches_go_to_the_device_of_the_tensors(seen, name):
    for index in (1, 0):
        CALLS[name][0](tensors(f"cuda:{index}"))
        assert seen.launched.pop() == index
    with pytest.raises(ValueError):
        CALLS[name][0](tensors("cuda:1"), stream=Stream(0x20, 0))
    assert not seen.launched


def test_tensors_of_other_devices_are_refused(seen):
    here, there = tensors("cuda:0"), tensors("cuda:1")
    i32 = torch.empty(4, dtype=torch.int32, device="cuda:1")
    half = lambda *shape: torch.empty(shape, dtype=torch.float16, device="cuda:1")
    for bad in (lambda: w4.rms_norm_quant(here.a, there.weight),
                lambda: w4.rms_norm_quant(here.a, here.weight, residual=there.a),
                lambda: w4.rms_norm_quant(here.a, here.weight, h=there.a),
                lambda: w4.rms_norm_quant(here.a, here.weight, a8=there.a8),
                lambda: w4.rms_norm_quant(here.a, here.weight, s_a=there.s_a),
                lambda: w4.silu_mul_quant(here.a, there.a),
                lambda: w4.silu_mul_quant(here.a, here.a, a8=there.a8),
                lambda: w4.silu_mul_quant(here.a, here.a, s_a=there.s_a),
                lambda: w4.rope_append(here.q, there.k, here.k, None, *here.kv),
                lambda: w4.rope_append(here.q, here.k, there.k, None, *here.kv),
                lambda: w4.rope_append(here.q, here.k, here.k, half(32, 64).float(), *here.kv),
                lambda: w4.rope_append(here.q, here.k, here.k, None, *here.kv, cu_q=i32),
                lambda: w4.rope_append(here.q, here.k, here.k, None, *here.kv, out=there.q),
                lambda: w4.paged_attention(here.q, *here.kv, cu_q=i32),
                lambda: w4.paged_attention(here.q, *here.kv, out=there.q),
                lambda: w4.paged_attention(here.q, *here.kv, workspace=there.blob),
                lambda: w4.paged_attention(here.q, *here.kv, workspace=torch.empty(8192, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    for i in range(4):
        kv = [*here.kv]
        kv[i] = there.kv[i]
        with pytest.raises(ValueError):
            w4.paged_attention(here.q, *kv)
        with pytest.raises(ValueError):
            w4.rope_append(here.q, here.k, here.k, None, *kv)
    assert not seen.launched
    # buffers that stay on the host, and a workspace with gaps
    with pytest.raises(ValueError):
        w4.rms_norm_quant(here.a, torch.empty(K, dtype=torch.float16))
    with pytest.raises(ValueError):
        w4.paged_attention(here.q, *here.kv, workspace=torch.empty((4096, 4), dtype=torch.uint8, device="cuda:0")[:, :2])
    assert not seen.launched
    assert w4.rms_norm_quant(here.a, here.weight, a8=here.a8)[1].shape == (M, K)
    assert len(seen.launched) == 1
