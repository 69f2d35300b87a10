"""The host side of the operators that verify and end a decoding step (no GPU):
argument validation, where calls allocate and launch, devices, sizes beyond 31
bits, and launch plans under sanitizers."""
import ctypes
import json
import os
import shutil
import subprocess
import sys

import pytest
import torch

import w4a8_gemm_amd as w4
import test_devices_host
import test_streams_host
from test_decoder_host import CSRC, FAKE, HERE, ROCM, ROOT, view
from test_streams_host import Stream

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
OTHER = 8192
streams_seen = test_streams_host.seen
devices_seen = test_devices_host.seen


# --------------------------------------------------------------- arguments
def statuses(call, cases):
    for kw, status in cases:
        assert call(**kw) == status, kw


def test_tree_mask_arguments():
    def call(parents=FAKE, lens=FAKE, cu=FAKE, batch=2, total=5, mask=FAKE, ld=1, words=1, positions=None):
        return w4.lib.w4a8_tree_mask(parents, lens, cu, batch, total, mask, ld, words, positions, None)
    statuses(call, [(dict(parents=None), 1), (dict(lens=None), 1), (dict(cu=None), 1), (dict(batch=-1), 1),
                    (dict(total=-1), 1), (dict(mask=None), 1), (dict(words=0), 1), (dict(words=2), 1),
                    (dict(batch=(1 << 22) + 1), 1), (dict(total=(1 << 22) + 1), 1), (dict(total=0), 0),
                    (dict(batch=0, total=0, lens=None, parents=None, mask=None), 0)])


def test_tree_attention_arguments():
    def call(v=None, q=FAKE, ldq=256, heads=4, mask=FAKE, ld=2, words=2, max_q=3, max_len=128, scale=0.1, window=0,
             out=FAKE, ldo=256, ws=None, ws_bytes=0):
        v = v or view(cu_q=FAKE, total_q=9)
        return w4.lib.w4a8_tree_attention(q, ldq, heads, ctypes.byref(v), mask, ld, words, max_q, max_len, scale, window,
                                          out, ldo, ws, ws_bytes, None)
    statuses(call, [(dict(q=None), 1), (dict(ldq=252), 1), (dict(out=FAKE + 2), 1), (dict(heads=3), 2), (dict(heads=0), 1),
                    (dict(window=-1), 1), (dict(scale=float("inf")), 1), (dict(max_len=-1), 1), (dict(max_q=-1), 1),
                    (dict(mask=None), 1), (dict(words=0), 1), (dict(words=3), 1), (dict(v=view(page_size=8)), 2),
                    (dict(v=view(batch=0, total_q=0), mask=None), 0), (dict(v=view(head_dim=72)), 2)])
    size = w4.lib.w4a8_tree_attention_workspace_size
    long = view(batch=1, cu_q=FAKE, total_q=8, max_pages=1000, block_table_ld=1000)
    need = size(ctypes.byref(long), 4, 8, 16000)
    assert need > 0                                    # a long sequence with few rows is split
    statuses(call, [(dict(v=long, max_len=16000), 3), (dict(v=long, max_len=16000, ws=FAKE, ws_bytes=need - 1), 3),
                    (dict(v=long, max_len=16000, ws=FAKE + 4, ws_bytes=need), 1)])
    assert size(ctypes.byref(long), 4, 8, 100) == 0 and size(ctypes.byref(view(page_size=8)), 4, 1, 16000) == 0


def test_accept_and_keep_arguments():
    def accept(drafted=FAKE, parents=FAKE, sampled=FAKE, lens=FAKE, cu=FAKE, batch=2, total=5, path=FAKE, ld=4, most=4,
               count=FAKE, tokens=FAKE, new=FAKE):
        return w4.lib.w4a8_tree_accept(drafted, parents, sampled, lens, cu, batch, total, path, ld, most, count, tokens,
                                       new, None)
    statuses(accept, [(dict(drafted=None), 1), (dict(parents=None), 1), (dict(sampled=None), 1), (dict(lens=None), 1),
                      (dict(cu=None), 1), (dict(path=None), 1), (dict(ld=3), 1), (dict(most=0), 1), (dict(count=None), 1),
                      (dict(tokens=None), 1), (dict(new=None), 1), (dict(batch=0, total=0), 0)])

    def keep(v=None, path=FAKE, ld=4, most=4, count=FAKE):
        return w4.lib.w4a8_kv_keep(ctypes.byref(v or view()), path, ld, most, count, None)
    statuses(keep, [(dict(path=None), 1), (dict(ld=3), 1), (dict(most=0), 1), (dict(count=None), 1),
                    (dict(v=view(page_size=8)), 2), (dict(v=view(data=None)), 1), (dict(v=view(batch=0, total_q=0)), 0),
                    (dict(v=view(batch=1 << 22, total_q=1 << 22, kv_heads=4096, page_stride=1 << 23, scale_stride=8192)), 2)])
    assert w4.lib.w4a8_kv_keep(None, FAKE, 4, 4, FAKE, None) == 1


def test_sample_arguments():
    def call(x=FAKE, f32=0, ld=100, rows=3, vocab=100, u=FAKE, s=(1.0, 0, 1.0, 0.0), tokens=FAKE, probs=None, dev=None,
             ws=None, ws_bytes=0):
        s = w4.Sampling(*s)
        for name in dev or ():
            setattr(s, name + "_dev", FAKE)
        return w4.lib.w4a8_sample(x, f32, ld, rows, vocab, u, ctypes.byref(s), tokens, probs, ws, ws_bytes, None)
    nan, inf = float("nan"), float("inf")
    statuses(call, [(dict(x=None), 1), (dict(x=FAKE + 1), 1), (dict(x=FAKE + 2, f32=1), 1), (dict(ld=99), 1),
                    (dict(rows=-1), 1), (dict(rows=(1 << 22) + 1), 1), (dict(vocab=0), 1), (dict(u=None), 1),
                    (dict(tokens=None), 1), (dict(s=(-1.0, 0, 1.0, 0.0)), 1), (dict(s=(nan, 0, 1.0, 0.0)), 1),
                    (dict(s=(inf, 0, 1.0, 0.0)), 1), (dict(s=(1.0, 0, nan, 0.0)), 1), (dict(s=(1.0, 0, 1.0, nan)), 1),
                    (dict(vocab=(1 << 19) + 1, ld=1 << 20), 2), (dict(rows=0, x=None), 0),
                    (dict(s=(nan, 0, 1.0, 0.0), dev=("temperature",), rows=0), 0)])
    assert w4.lib.w4a8_sample(FAKE, 0, 100, 3, 100, FAKE, None, FAKE, None, None, 0, None) == 1
    need = w4.lib.w4a8_sample_workspace_size(0, 3, 50000)
    assert need > 0 and w4.lib.w4a8_sample_workspace_size(0, 3, 100) == 0
    assert w4.lib.w4a8_sample_workspace_size(0, 3, 1 << 20) == 0 and w4.lib.w4a8_sample_workspace_size(0, -3, 50000) == 0
    long = dict(vocab=50000, ld=50000)
    statuses(call, [(long, 3), (dict(**long, ws=FAKE, ws_bytes=need - 1), 3), (dict(**long, ws_bytes=need), 1),
                    (dict(**long, ws=FAKE + 8, ws_bytes=need), 1)])


def test_page_arguments():
    def fork(table=FAKE, ld=8, width=8, lens=FAKE, batch=3, refs=FAKE, pages=10, page=16, parent=FAKE, rows=4, new=OTHER,
             new_ld=8, new_lens=OTHER, new_refs=OTHER):
        return w4.lib.w4a8_kv_fork(table, ld, width, lens, batch, refs, pages, page, parent, rows, new, new_ld, new_lens,
                                   new_refs, None)
    same = [(dict(table=None), 1), (dict(ld=7), 1), (dict(width=0), 1), (dict(lens=None), 1), (dict(batch=-1), 1),
            (dict(refs=None), 1), (dict(pages=0), 1), (dict(page=24), 2), (dict(page=2048), 2), (dict(new=None), 1),
            (dict(new=FAKE), 1), (dict(new_ld=7), 1), (dict(new_lens=None), 1), (dict(new_lens=FAKE), 1),
            (dict(new_refs=None), 1), (dict(new_refs=FAKE), 1), (dict(pages=(1 << 22) + 1), 2),
            (dict(width=1 << 20, ld=1 << 20, new_ld=1 << 20, batch=1 << 12), 2),
            (dict(width=1 << 27, ld=1 << 27, new_ld=1 << 27), 1)]
    statuses(fork, same + [(dict(parent=None), 1), (dict(rows=-1), 1)])

    def alloc(table=FAKE, ld=8, width=8, lens=FAKE, batch=3, refs=FAKE, pages=10, page=16, tokens=None, each=1, new=OTHER,
              new_ld=8, new_lens=OTHER, new_refs=OTHER, src=FAKE, dst=FAKE, counts=FAKE, ws=FAKE, ws_bytes=None):
        need = w4.lib.w4a8_kv_alloc_workspace_size(batch, pages)
        return w4.lib.w4a8_kv_alloc(table, ld, width, lens, batch, refs, pages, page, tokens, each, new, new_ld, new_lens,
                                    new_refs, src, dst, counts, ws, need if ws_bytes is None else ws_bytes, None)
    statuses(alloc, same + [(dict(src=None), 1), (dict(dst=None), 1), (dict(counts=None), 1), (dict(each=-1), 1),
                            (dict(ws_bytes=20), 3), (dict(ws=None), 1), (dict(ws=FAKE + 4), 1)])

    def compact(table=FAKE, ld=8, width=8, batch=3, refs=FAKE, pages=10, new=OTHER, new_ld=8, new_refs=OTHER, place=FAKE,
                src=FAKE, dst=FAKE, counts=FAKE, ws=FAKE, ws_bytes=None):
        need = w4.lib.w4a8_kv_compact_workspace_size(pages)
        return w4.lib.w4a8_kv_compact(table, ld, width, batch, refs, pages, new, new_ld, new_refs, place, src, dst, counts,
                                      ws, need if ws_bytes is None else ws_bytes, None)
    statuses(compact, [(kw, st) for kw, st in same if not {"lens", "page", "new_lens"} & set(kw) and kw.get("width") != 1 << 27]
             + [(dict(place=None), 1), (dict(src=None), 1), (dict(dst=None), 1), (dict(counts=None), 1),
                (dict(ws_bytes=4), 3), (dict(ws=None), 1)])

    def copy(data=FAKE, scale=FAKE, stride=4096, scale_stride=4, pages=4, page=16, heads=2, dim=64, src=FAKE, dst=FAKE,
             pairs=3, count=None):
        return w4.lib.w4a8_kv_copy_pages(data, scale, stride, scale_stride, pages, page, heads, dim, src, dst, pairs, count,
                                         None)
    statuses(copy, [(dict(data=None), 1), (dict(data=FAKE + 8), 1), (dict(scale=None), 1), (dict(stride=4080), 1),
                    (dict(stride=4104), 1), (dict(scale_stride=3), 1), (dict(pages=0), 1), (dict(page=8), 2),
                    (dict(heads=0), 1), (dict(heads=5000), 2), (dict(dim=72), 2), (dict(dim=272), 2), (dict(src=None), 1),
                    (dict(dst=None), 1), (dict(pairs=-1), 1), (dict(pairs=0, src=None), 0),
                    (dict(heads=4096, page=1024, dim=256, stride=1 << 31, scale_stride=8192), 2)])


# ------------------------------------------------------- streams and devices
def tensors(device="cuda:0"):
    t = test_streams_host.tensors(device)
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=device)
    f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=device)
    t.nodes, t.cu, t.mask, t.path, t.count, t.refs, t.u = i32(3), i32(4), i32(3, 1), i32(3, 2), i32(3), i32(9), f32(5)
    t.cos_sin, t.five = f32(40, 64), i32(5)
    return t


# name -> (call, buffers it allocates, tensors it returns)
CALLS = {
    "tree_mask": (lambda t, **kw: w4.tree_mask(t.nodes, t.kv[3], cu_q=t.cu, **kw), 2, 2),
    "tree_mask, given": (lambda t, **kw: w4.tree_mask(t.nodes, t.kv[3], mask=t.mask, positions=t.count, **kw), 0, 0),
    "tree_attention": (lambda t, **kw: w4.tree_attention(t.q, *t.kv, t.mask, **kw), 2, 1),
    "tree_accept": (lambda t, **kw: w4.tree_accept(t.nodes, t.nodes, t.nodes, t.kv[3], **kw), 4, 4),
    "kv_keep": (lambda t, **kw: w4.kv_keep(*t.kv, t.path, t.count, **kw), 0, 0),
    "sample": (lambda t, **kw: w4.sample(t.a, t.u, **kw), 3, 2),
    "sample, settings": (lambda t, **kw: w4.sample(t.a.float(), t.u, t.u, top_p=t.u, probs=t.u, **kw), 2, 1),
    "sample, given": (lambda t, **kw: w4.sample(t.a, t.u, tokens=t.five, probs=t.u, workspace=t.blob, **kw), 0, 0),
    "kv_fork": (lambda t, **kw: w4.kv_fork(t.kv[2], t.kv[3], t.refs, t.nodes, 16, **kw), 3, 3),
    "kv_alloc": (lambda t, **kw: w4.kv_alloc(t.kv[2], t.kv[3], t.refs, 1, 16, **kw), 7, 6),
    "kv_compact": (lambda t, **kw: w4.kv_compact(t.kv[2], t.refs, **kw), 7, 6),
    "kv_copy_pages": (lambda t, **kw: w4.kv_copy_pages(t.kv[0], t.kv[1], t.nodes, t.nodes, t.count, **kw), 0, 0),
    "rope_append, positions": (lambda t, **kw: w4.rope_append(t.q, t.k, t.k, t.cos_sin, *t.kv, positions=t.nodes, **kw),
                               1, 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_buffers_come_from_the_stream_they_are_used_on(streams_seen, name):
    call, allocated, returned = CALLS[name]
    t = tensors()
    streams_seen.empty.clear()
    out = call(t, stream=Stream(0x20))
    assert streams_seen.launched == [0x20]
    assert streams_seen.empty == [0x20] * allocated
    out = out if isinstance(out, tuple) else (out,)
    assert len(streams_seen.recorded) == returned and all(s == 0x10 for _, s in streams_seen.recorded)
    assert {i for i, _ in streams_seen.recorded} <= {id(t) for t in out}


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_by_default(streams_seen, name):
    call, allocated, _ = CALLS[name]
    t = tensors()
    streams_seen.empty.clear()
    call(t)
    assert streams_seen.launched == [0x10] and streams_seen.empty == [0x10] * allocated and not streams_seen.recorded


@pytest.mark.parametrize("name", CALLS)
def test_launches_go_to_the_device_of_the_tensors(devices_seen, name):
    for index in (1, 0):
        CALLS[name][0](tensors(f"cuda:{index}"))
        assert devices_seen.launched.pop() == index
    with pytest.raises(ValueError):
        CALLS[name][0](tensors("cuda:1"), stream=Stream(0x20, 0))
    assert not devices_seen.launched


def test_tensors_that_do_not_fit_are_refused(devices_seen):
    """Of another device, on the host, of another type or shape."""
    here, there = tensors("cuda:0"), tensors("cuda:1")
    wide = torch.empty((3, 8), dtype=torch.int32, device="cuda:0")[:, ::2]
    long = lambda *shape: torch.empty(shape, dtype=torch.int64, device="cuda:0")
    for bad in (lambda: w4.tree_mask(here.nodes, there.kv[3]), lambda: w4.tree_mask(here.nodes, here.kv[3], cu_q=there.cu),
                lambda: w4.tree_mask(here.nodes, here.kv[3], mask=there.mask),
                lambda: w4.tree_mask(here.nodes, here.kv[3], positions=there.count),
                lambda: w4.tree_mask(here.refs, here.kv[3]), lambda: w4.tree_mask(long(3), here.kv[3]),
                lambda: w4.tree_mask(here.nodes, here.kv[3], cu_q=here.nodes),
                lambda: w4.tree_attention(here.q, *here.kv, there.mask), lambda: w4.tree_attention(here.q, *here.kv, long(3, 1)),
                lambda: w4.tree_attention(here.q, *here.kv, wide), lambda: w4.tree_attention(here.q, *here.kv, here.mask[:2]),
                lambda: w4.tree_attention(here.q, *here.kv, here.mask[:, :0]),
                lambda: w4.tree_attention(here.q, *here.kv, here.mask, out=there.q),
                lambda: w4.tree_attention(here.q, *here.kv, here.mask, workspace=there.blob),
                lambda: w4.tree_accept(here.nodes, there.nodes, here.nodes, here.kv[3]),
                lambda: w4.tree_accept(here.nodes, here.nodes, there.nodes, here.kv[3]),
                lambda: w4.tree_accept(here.refs, here.nodes, here.nodes, here.kv[3]),
                lambda: w4.kv_keep(*here.kv, there.path, here.count), lambda: w4.kv_keep(*here.kv, here.path, there.count),
                lambda: w4.kv_keep(*here.kv, here.path[:2], here.count), lambda: w4.kv_keep(*here.kv, wide, here.count[:2]),
                lambda: w4.sample(here.a, there.u), lambda: w4.sample(here.a8, here.u), lambda: w4.sample(here.a, here.u[:4]),
                lambda: w4.sample(here.a, here.u, there.u), lambda: w4.sample(here.a, here.u, top_k=here.u),
                lambda: w4.sample(here.a, here.u, top_p=here.u[:2]), lambda: w4.sample(here.a, here.u, tokens=here.nodes),
                lambda: w4.sample(here.a, here.u, probs=there.u), lambda: w4.sample(here.a.t(), here.u),
                lambda: w4.sample(here.a.double(), here.u), lambda: w4.sample(here.a, here.u, workspace=there.blob),
                lambda: w4.kv_fork(here.kv[2], there.kv[3], here.refs, here.nodes, 16),
                lambda: w4.kv_fork(here.kv[2], here.kv[3], there.refs, here.nodes, 16),
                lambda: w4.kv_fork(here.kv[2], here.kv[3], here.refs, there.nodes, 16),
                lambda: w4.kv_fork(long(3, 8), here.kv[3], here.refs, here.nodes, 16),
                lambda: w4.kv_alloc(here.kv[2], here.kv[3], here.refs, there.nodes, 16),
                lambda: w4.kv_alloc(here.kv[2], here.kv[3], here.refs, -1, 16),
                lambda: w4.kv_alloc(here.kv[2], here.kv[3], here.refs, 1 << 31, 16),
                lambda: w4.kv_alloc(here.kv[2], here.kv[3], there.refs, 1, 16),
                lambda: w4.kv_compact(here.kv[2], there.refs), lambda: w4.kv_compact(here.refs, here.refs),
                lambda: w4.kv_copy_pages(here.kv[0], there.kv[1], here.nodes, here.nodes),
                lambda: w4.kv_copy_pages(here.kv[0], here.kv[1], there.nodes, here.nodes),
                lambda: w4.kv_copy_pages(here.kv[0], here.kv[1], here.nodes, here.refs),
                lambda: w4.kv_copy_pages(here.kv[0], here.kv[1], here.nodes, here.nodes, there.count),
                lambda: w4.kv_copy_pages(here.kv[0], here.kv[1], here.nodes, here.nodes, long(1)),
                lambda: w4.rope_append(here.q, here.k, here.k, None, *here.kv, positions=there.nodes),
                lambda: w4.rope_append(here.q, here.k, here.k, None, *here.kv, positions=here.refs),
                lambda: w4.tree_mask(torch.empty(3, dtype=torch.int32), here.kv[3]),
                lambda: w4.sample(torch.empty(5, 8), torch.empty(5)),
                lambda: w4.kv_copy_pages(torch.empty(9, 2, 2, 16, 64, dtype=torch.int8), here.kv[1], here.nodes, here.nodes)):
        with pytest.raises(ValueError):
            bad()
    assert not devices_seen.launched


def test_sizes_beyond_the_c_interface(devices_seen):
    big = 2 ** 32
    far = lambda shape, stride, dtype: torch.empty_strided(shape, stride, dtype=dtype, device="cuda:0")
    t = tensors()
    mask, table = far((3, 1), (big, 1), torch.int32), far((3, 8), (big + 8, 1), torch.int32)
    for bad in (lambda: w4.tree_attention(t.q, *t.kv, mask), lambda: w4.sample(far((5, 64), (big, 1), torch.float16), t.u),
                lambda: w4.kv_fork(table, t.kv[3], t.refs, t.nodes, 16), lambda: w4.kv_compact(table, t.refs),
                lambda: w4.kv_keep(*t.kv, far((3, 2), (big, 1), torch.int32), t.count),
                lambda: w4.kv_compact(t.kv[2], far((big,), (1,), torch.int32))):
        with pytest.raises(ValueError):
            bad()
    assert not devices_seen.launched
    w4.tree_attention(t.q, *t.kv, t.mask, max_q=big + 1, max_len=big + 5, window=big + 5)
    w4.sample(t.a, t.u, top_k=big)
    assert len(devices_seen.launched) == 2


# --------------------------------------------------------------- sanitizers
@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_abi_under_asan_and_ubsan(tmp_path):
    flags = ["-O1", "-g", "-fPIC", "-std=c++17", "-fno-omit-frame-pointer",
             "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
             "-I", os.path.join(ROCM, "include"), "-I", os.path.join(ROOT, "include")]
    objs = []
    for src in (os.path.join(CSRC, "verify_api.cpp"), os.path.join(HERE, "host_stubs_verify.cpp")):
        obj = os.path.join(str(tmp_path), os.path.basename(src) + ".o")
        subprocess.run(["g++", *flags, "-x", "c++", "-c", src, "-o", obj], check=True)
        objs.append(obj)
    lib = os.path.join(str(tmp_path), "libverify_host.so")
    subprocess.run(["g++", "-shared", "-fsanitize=address,undefined", *objs, "-o", lib], check=True)
    asan = subprocess.run(["g++", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, os.path.join(HERE, "san_driver_verify.py"), lib],
                         capture_output=True, text=True, env=env, timeout=600)
    assert res.returncode == 0, res.stdout[-2000:] + res.stderr[-4000:]
    seen = json.loads(res.stdout.strip().splitlines()[-1])
    for name, status in seen.items():
        assert 1 in status and 7 in status, (name, status)       # refused, and reached a launch
    assert all(2 in seen[name] for name in ("attention", "keep", "sample", "fork", "alloc", "compact", "copy"))
    assert all(3 in seen[name] for name in ("attention", "sample", "alloc", "compact"))
