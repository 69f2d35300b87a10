"""The host side of the decoder-layer operators (no GPU): argument validation,
launch plans under sanitizers, and the rotary table."""
import ctypes
import json
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import w4a8_gemm_amd as w4

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "w4a8_gemm_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
FAKE = 4096            # never dereferenced: rejected first


def view(**kw):
    v = dict(data=FAKE, scale=FAKE, page_stride=2 * 2 * 16 * 64, scale_stride=4, num_pages=4, page_size=16,
             kv_heads=2, head_dim=64, block_table=FAKE, block_table_ld=8, max_pages=8, seq_lens=FAKE,
             cu_q=None, batch=3, total_q=3)
    v.update(kw)
    return w4.KvView(*(v[name] for name, _ in w4.KvView._fields_))


def append(v, q=FAKE, ldq=256, k=FAKE, ldk=128, cos=FAKE, rotary=64, max_pos=100, heads=4, out=FAKE, ldo=256):
    return w4.lib.w4a8_rope_append(q, ldq, k, ldk, FAKE, 128, heads, cos, rotary, max_pos, 0,
                                   ctypes.byref(v) if v else None, out, ldo, None)


def attend(v, q=FAKE, ldq=256, heads=4, max_q=1, max_len=128, scale=0.1, window=0, out=FAKE, ldo=256,
           ws=None, ws_bytes=0):
    return w4.lib.w4a8_paged_attention(q, ldq, heads, ctypes.byref(v) if v else None, max_q, max_len,
                                       scale, window, out, ldo, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(data=None), 1), (dict(scale=None), 1), (dict(block_table=None), 1), (dict(seq_lens=None), 1),
    (dict(data=FAKE + 8), 1), (dict(num_pages=0), 1), (dict(kv_heads=0), 1), (dict(batch=-1), 1),
    (dict(total_q=-1), 1), (dict(total_q=2), 1),                    # no cu_q: one token each
    (dict(max_pages=0), 1), (dict(block_table_ld=7), 1), (dict(page_stride=4095), 1),
    (dict(page_stride=4104), 1), (dict(scale_stride=3), 1), (dict(max_pages=1 << 27, block_table_ld=1 << 27), 1),
    (dict(page_size=8), 2), (dict(page_size=24), 2), (dict(page_size=2048), 2),
    (dict(head_dim=72), 2), (dict(head_dim=272), 2), (dict(head_dim=0), 2), (dict(kv_heads=5000), 2),
    (dict(batch=0, total_q=0), 0), (dict(cu_q=FAKE, total_q=0), 0),
])
def test_view_is_checked(change, status):
    assert append(view(**change)) == status
    assert attend(view(**change)) == status


def test_append_arguments():
    v = view()
    for kw, status in ((dict(q=None), 1), (dict(q=FAKE + 8), 1), (dict(ldq=255), 1), (dict(ldq=260), 1),
                       (dict(k=None), 1), (dict(ldk=120), 1), (dict(out=None), 1), (dict(ldo=248), 1),
                       (dict(rotary=-16), 1), (dict(rotary=80), 1), (dict(rotary=24), 2),
                       (dict(cos=None), 1), (dict(cos=FAKE + 4), 1), (dict(max_pos=0), 1), (dict(heads=0), 1),
                       (dict(heads=5000), 2)):
        assert append(v, **kw) == status, kw
    assert append(None) == 1


def test_attention_arguments_and_workspace():
    v = view()
    for kw, status in ((dict(q=None), 1), (dict(ldq=252), 1), (dict(out=FAKE + 2), 1), (dict(heads=3), 2),
                       (dict(heads=0), 1), (dict(window=-1), 1), (dict(scale=float("inf")), 1),
                       (dict(max_len=-1), 1), (dict(max_q=-1), 1)):
        assert attend(v, **kw) == status, kw
    assert attend(None) == 1
    size = w4.lib.w4a8_paged_attention_workspace_size
    one = view(batch=1, total_q=1, max_pages=1000, block_table_ld=1000)
    need = size(ctypes.byref(one), 4, 1, 16000)
    assert need > 0                                    # a long sequence with few rows is split
    assert attend(one, max_len=16000) == 3
    assert attend(one, max_len=16000, ws=FAKE, ws_bytes=need - 1) == 3
    assert attend(one, max_len=16000, ws=FAKE + 4, ws_bytes=need) == 1
    assert size(ctypes.byref(one), 4, 1, 100) == 0     # a short one is not
    assert size(ctypes.byref(view(page_size=8)), 4, 1, 16000) == 0
    many = view(cu_q=FAKE, batch=8, total_q=40000)
    assert size(ctypes.byref(many), 4, 5000, 5000) == 0   # row tiles alone fill the device


def test_row_operator_arguments():
    L = w4.lib
    norm = lambda x=FAKE, ldx=64, r=None, ldr=0, w=FAKE, eps=1e-5, m=4, k=64, h=None, ldh=0, a=FAKE, lda=64, s=FAKE: \
        L.w4a8_rms_norm_quant(x, ldx, r, ldr, w, eps, m, k, h, ldh, a, lda, s, None)
    for kw in (dict(x=None), dict(ldx=63), dict(w=None), dict(m=-1), dict(k=0), dict(a=None), dict(lda=10),
               dict(s=None), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(r=FAKE, ldr=64), dict(r=FAKE, ldr=60, h=FAKE, ldh=64), dict(h=FAKE, ldh=63),
               dict(m=(1 << 22) + 1), dict(k=(1 << 30) + 1, ldx=2 ** 31 - 1, lda=2 ** 31 - 1)):
        assert norm(**kw) == 1, kw
    assert norm(m=0) == 0
    silu = lambda g=FAKE, ldg=64, u=FAKE, ldu=64, m=4, k=64, a=FAKE, lda=64, s=FAKE: \
        L.w4a8_silu_mul_quant(g, ldg, u, ldu, m, k, a, lda, s, None)
    for kw in (dict(g=None), dict(u=None), dict(a=None), dict(s=None), dict(ldg=60), dict(ldu=60),
               dict(lda=60), dict(m=-2), dict(k=0), dict(m=(1 << 22) + 1)):
        assert silu(**kw) == 1, kw
    assert silu(m=0) == 0


def test_rope_table():
    t = w4.rope_table(50, 64, device="cpu")
    assert t.shape == (50, 64) and t.dtype == torch.float32
    i, pos = np.arange(32), np.arange(50)[:, None]
    angle = pos * 10000.0 ** (-2.0 * i / 64)
    # computed in 64 bits and rounded once
    assert (np.abs(t[:, :32].numpy() - np.cos(angle)) <= 2.0 ** -24).all()
    assert (np.abs(t[:, 32:].numpy() - np.sin(angle)) <= 2.0 ** -24).all()
    linear = w4.rope_table(50, 64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(linear[::4], t[:13])            # position 4p turns as p did
    based = w4.rope_table(50, 64, scaling="base", factor=8.0, device="cpu").double()
    assert torch.allclose(based[:, 0], t[:, 0].double(), atol=1e-6)        # the highest frequency stays
    lowest = 10000.0 ** (-62 / 64) / 8.0
    assert abs(float(based[49, 63]) - np.sin(49 * lowest)) < 1e-7          # the lowest is divided
    bands = w4.rope_table(50, 64, scaling="bands", factor=8.0, original_max_pos=2048, device="cpu").double()
    turns = 2048 * 10000.0 ** (-2.0 * i / 64) / (2 * np.pi)
    assert torch.allclose(bands[:, :32][:, turns > 4], t[:, :32].double()[:, turns > 4], atol=1e-6)
    slow = np.flatnonzero(turns < 1)
    assert np.allclose(bands[49, 32 + slow].numpy(), np.sin(49 * 10000.0 ** (-2.0 * slow / 64) / 8.0), atol=1e-7)
    for bad in (dict(rotary_dim=63), dict(max_pos=0), dict(factor=0.0), dict(scaling="other"),
                dict(scaling="bands", low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            w4.rope_table(**{"max_pos": 8, "rotary_dim": 64, "device": "cpu", **bad})


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_decoder_abi_under_asan_and_ubsan(tmp_path):
    flags = ["-O1", "-g", "-fPIC", "-std=c++17", "-fno-omit-frame-pointer",
             "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
             "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include")]
    objs = []
    for src in (os.path.join(CSRC, "decoder_api.cpp"), os.path.join(HERE, "host_stubs_decoder.cpp")):
        obj = os.path.join(str(tmp_path), os.path.basename(src) + ".o")
        subprocess.run(["g++", *flags, "-x", "c++", "-c", src, "-o", obj], check=True)
        objs.append(obj)
    lib = os.path.join(str(tmp_path), "libdecoder_host.so")
    subprocess.run(["g++", "-shared", "-fsanitize=address,undefined", *objs, "-o", lib], check=True)
    asan = subprocess.run(["g++", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, os.path.join(HERE, "san_driver_decoder.py"), lib],
                         capture_output=True, text=True, env=env, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    seen = json.loads(res.stdout.strip().splitlines()[-1])
    for name, statuses in seen.items():
        assert 1 in statuses and 7 in statuses, (name, statuses)   # refused, and reached a launch
    assert 2 in seen["append"] and 2 in seen["attention"] and 3 in seen["attention"]
