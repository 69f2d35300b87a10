"""Python binding of libw4a8.so (the MI355X W4A8 linear layer).

This module only marshals arguments: numpy arrays for the host packer,
torch tensors for device memory, and torch's current HIP stream.  Every
step of the layer runs inside the C ABI library; there is no fallback.  If
the library has not been built, importing this module raises.

    blob  = pack(w, g)                       # host, offline
    wdev  = to_device(blob)                  # one copy to HBM
    a8, s_a = quant_act(a)                   # per-token int8 (GPU)
    y     = gemm(a8, s_a, wdev, n, k, g)     # W4A8 GEMM (GPU)

GPU calls run on the device of their tensors, all on one, and take stream=, a
torch.cuda.Stream of it to launch on (default: the current one); that the inputs
are ready there is the caller's to arrange.

Between the linears of a decoder: rms_norm_quant, silu_mul_quant, and a paged
int8 KV cache (kv_cache, rope_table, rope_append, paged_attention).  Its pages are
handed out, shared, freed and moved by kv_alloc, kv_fork, kv_compact and
kv_copy_pages.

At the end of a step: sample.  For drafted token trees: tree_mask,
tree_attention, tree_accept, kv_keep.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import re

import numpy as np
# torch is imported before the library is loaded: it carries its own HIP runtime
# (same soname as the system one).  Loading it first makes the library's
# libamdhip64 dependency resolve to that already-loaded runtime, so torch
# allocations, torch streams and this library's kernels share one HIP runtime
# in the process.
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a8.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "w4a8.h")

GROUP_PER_CHANNEL = 0
K_QUANTUM = 128
N_QUANTUM = 16
K_MAX = 131072
M_MAX = 1 << 22

STATUS = {
    0: "W4A8_OK",
    1: "W4A8_ERR_INVALID_ARGUMENT",
    2: "W4A8_ERR_UNSUPPORTED",
    3: "W4A8_ERR_BUFFER_TOO_SMALL",
    4: "W4A8_ERR_NONFINITE",
    5: "W4A8_ERR_RANGE",
    6: "W4A8_ERR_LAYOUT",
    7: "W4A8_ERR_DEVICE",
}


class W4A8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class GemmOpts(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("k_split", ctypes.c_int),
                ("n_tiles", ctypes.c_int), ("m_tiles", ctypes.c_int),
                ("stages", ctypes.c_int), ("row_groups", ctypes.c_int),
                ("slices", ctypes.c_int), ("workgroups", ctypes.c_int)]


class KvView(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_longlong), ("scale_stride", ctypes.c_longlong),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("block_table", ctypes.c_void_p), ("block_table_ld", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("seq_lens", ctypes.c_void_p),
                ("cu_q", ctypes.c_void_p), ("batch", ctypes.c_int), ("total_q", ctypes.c_int)]


class Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("temperature_dev", ctypes.c_void_p),
                ("top_k_dev", ctypes.c_void_p), ("top_p_dev", ctypes.c_void_p),
                ("min_p_dev", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python w4a8_gemm_amd/build.py` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong
    sig = {
        "w4a8_status_string": (ctypes.c_char_p, [I]),
        "w4a8_last_device_error": (ctypes.c_char_p, []),
        "w4a8_packed_size": (Z, [I, I, I]),
        "w4a8_pack": (I, [P, I, I, I, I, P, Z, I]),
        "w4a8_blob_info": (I, [P, Z, P, P, P]),
        "w4a8_unpack": (I, [P, Z, P, P, P, P]),
        "w4a8_quant_act": (I, [P, I, I, I, P, I, P, P]),
        "w4a8_quant_act_static": (I, [P, I, I, I, ctypes.c_uint16, P, I, P, P]),
        "w4a8_gemm_workspace_size": (Z, [I, I, I, I, P]),
        "w4a8_gemm": (I, [P, I, P, I, P, I, I, I, P, I, P, I, P, Z, P, P]),
        "w4a8_linear": (I, [P, I, I, I, P, I, I, P, I, P, I, P, P, I, P, Z, P, P]),
        "w4a8_linear_launches": (I, [I, I, I, I, P]),
        "w4a16_gemm": (I, [P, I, I, I, P, I, I, P, I, P, P]),
        "w4a8_read_probe": (I, [P, Z, I, P, P]),
        "w4a8_rms_norm_quant": (I, [P, I, P, I, P, ctypes.c_float, I, I, P, I, P, I, P, P]),
        "w4a8_silu_mul_quant": (I, [P, I, P, I, I, I, P, I, P, P]),
        "w4a8_rope_append": (I, [P, I, P, I, P, I, I, P, I, I, I, P, P, I, P]),
        "w4a8_paged_attention_workspace_size": (Z, [P, I, I, I]),
        "w4a8_paged_attention": (I, [P, I, I, P, I, I, ctypes.c_float, I, P, I, P, Z, P]),
        "w4a8_rope_append_at": (I, [P, I, P, I, P, I, I, P, I, I, I, P, P, P, I, P]),
        "w4a8_tree_mask": (I, [P, P, P, I, I, P, I, I, P, P]),
        "w4a8_tree_attention_workspace_size": (Z, [P, I, I, I]),
        "w4a8_tree_attention": (I, [P, I, I, P, P, I, I, I, I, ctypes.c_float, I, P, I, P, Z, P]),
        "w4a8_tree_accept": (I, [P, P, P, P, P, I, I, P, I, I, P, P, P, P]),
        "w4a8_kv_keep": (I, [P, P, I, I, P, P]),
        "w4a8_sample_workspace_size": (Z, [I, I, I]),
        "w4a8_sample": (I, [P, I, I, I, I, P, P, P, P, P, Z, P]),
        "w4a8_kv_fork": (I, [P, I, I, P, I, P, I, I, P, I, P, I, P, P, P]),
        "w4a8_kv_alloc_workspace_size": (Z, [I, I]),
        "w4a8_kv_alloc": (I, [P, I, I, P, I, P, I, I, P, I, P, I, P, P, P, P, P, P, Z, P]),
        "w4a8_kv_compact_workspace_size": (Z, [I]),
        "w4a8_kv_compact": (I, [P, I, I, I, P, I, P, I, P, P, P, P, P, P, Z, P]),
        "w4a8_kv_copy_pages": (I, [P, P, L, L, I, I, I, I, P, P, I, P, P]),
        "w4a8_gemm_noalloc": (I, [P, I, P, I, P, I, I, I, P, I, P, I, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def header_functions() -> list[str]:
    """Names of the functions declared in include/w4a8.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"\b(w4a8_[a-z0-9_]+)\s*\(", text)))


def _check(status: int, where: str):
    if status != 0:
        if status == 7:
            where = f"{where} ({lib.w4a8_last_device_error().decode()})"
        raise W4A8Error(status, where)


def status_string(status: int) -> str:
    return lib.w4a8_status_string(status).decode()


# ------------------------------------------------------------------ host side
GROUP_PER_CHANNEL = 0
CODEBOOK_NF = 1      # g value of the non-uniform codebook mode


def packed_size(n: int, k: int, g: int) -> int:
    return int(lib.w4a8_packed_size(n, k, g))


def pack(w: np.ndarray, g: int, n_threads: int = 0) -> np.ndarray:
    """Quantize and pack an N x K float32 weight matrix; returns the blob (uint8)."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    n, k = w.shape
    size = packed_size(n, k, g)
    if size == 0:
        raise W4A8Error(2, "w4a8_packed_size")
    blob = np.empty(size, dtype=np.uint8)
    _check(lib.w4a8_pack(w.ctypes.data, n, k, k, g, blob.ctypes.data, size, n_threads),
           "w4a8_pack")
    return blob


def blob_info(blob: np.ndarray) -> tuple[int, int, int]:
    n, k, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib.w4a8_blob_info(blob.ctypes.data, blob.nbytes, ctypes.byref(n), ctypes.byref(k),
                              ctypes.byref(g)), "w4a8_blob_info")
    return n.value, k.value, g.value


def unpack(blob: np.ndarray) -> dict:
    """Logical arrays of a host blob: q [N,K], z/s2 [N,G], s1 [N] (float16)."""
    n, k, g = blob_info(blob)
    groups = 1 if g == 0 else (0 if g == CODEBOOK_NF else k // g)
    q = np.empty((n, k), dtype=np.uint8)
    z = np.empty((n, groups), dtype=np.uint8)
    s2 = np.empty((n, groups), dtype=np.uint8)
    s1 = np.empty(n, dtype=np.uint16)
    _check(lib.w4a8_unpack(blob.ctypes.data, blob.nbytes, q.ctypes.data, z.ctypes.data,
                           s2.ctypes.data, s1.ctypes.data), "w4a8_unpack")
    out = {"q": q, "z": z, "s2": s2, "s1": s1.view(np.float16), "n": n, "k": k, "g": g}
    if g == CODEBOOK_NF:
        out["levels"] = blob[56:72].view(np.int8).astype(np.int32)
    return out


# ------------------------------------------------------------------ device side
def _stream_of(t, stream=None) -> int:
    """The given stream, or the current one of t's device."""
    if stream is not None:
        return int(stream.cuda_stream)
    # the raw handle where torch offers it: a Stream object takes 2.9 us to make
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(t.device.index) if raw else int(torch.cuda.current_stream(t.device).cuda_stream)


def _on_device(fn):
    """Runs fn(t, ...) with the device of its first tensor current, since that is
    where a launch goes, and refuses a stream of another device."""
    params = list(inspect.signature(fn).parameters)
    at = params.index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        index = (args[0] if args else kw[params[0]]).get_device()
        if index < 0:
            return fn(*args, **kw)          # fn refuses it
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is not None and stream.device.index != index:
            raise ValueError(f"stream: expected one of cuda:{index}, got one of {stream.device}")
        if index == torch.cuda.current_device():
            return fn(*args, **kw)
        with torch.cuda.device(index):
            return fn(*args, **kw)
    return call


def _empty(shape, dtype, device, stream, returned=True):
    """A buffer for a call that launches on `stream` (None: the current one),
    from that stream's pool: memory of the current stream may still be in use
    by work queued there.  One that is returned is marked as used by the current
    stream too, where it will be read, so that its memory is not given out again
    before that is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    caller = torch.cuda.current_stream()
    torch.cuda.set_stream(stream)        # both of the current device; a
    try:                                 # torch.cuda.stream() takes 5 us more
        t = torch.empty(shape, dtype=dtype, device=device)
    finally:
        torch.cuda.set_stream(caller)
    if returned:
        t.record_stream(caller)
    return t


def to_device(blob: np.ndarray, device="cuda"):
    """Copy a packed blob to device memory (a uint8 torch tensor)."""
    return torch.from_numpy(blob).to(device)


@_on_device
def quant_act(a, a8=None, s_a=None, stream=None):
    """Per-token int8 quantization of an M x K float16 CUDA tensor."""
    assert a.dtype == torch.float16 and a.is_cuda and a.dim() == 2 and a.stride(1) == 1
    m, k = a.shape
    if a8 is None:
        a8 = _empty((m, k), torch.int8, a.device, stream)
    if s_a is None:
        s_a = _empty((m,), torch.float16, a.device, stream)
    _check(lib.w4a8_quant_act(a.data_ptr(), m, k, a.stride(0), a8.data_ptr(), a8.stride(0),
                              s_a.data_ptr(), _stream_of(a, stream)), "w4a8_quant_act")
    return a8, s_a


@_on_device
def quant_act_static(a, scale, a8=None, s_a=None, stream=None):
    """Int8 quantization of an M x K float16 CUDA tensor with one static
    fp16 scale; s_a is filled with the scale for every row."""
    assert a.dtype == torch.float16 and a.is_cuda and a.dim() == 2 and a.stride(1) == 1
    m, k = a.shape
    if a8 is None:
        a8 = _empty((m, k), torch.int8, a.device, stream)
    if s_a is None:
        s_a = _empty((m,), torch.float16, a.device, stream)
    bits = int(np.array([scale], dtype=np.float16).view(np.uint16)[0])
    _check(lib.w4a8_quant_act_static(a.data_ptr(), m, k, a.stride(0), bits, a8.data_ptr(),
                                     a8.stride(0), s_a.data_ptr(), _stream_of(a, stream)),
           "w4a8_quant_act_static")
    return a8, s_a


@_on_device
def gemm(a8, s_a, blob_dev, n: int, k: int, g: int, y=None, acc=None, want_acc=False,
         variant: int = 0, k_split: int = 0, n_tiles: int = 0, m_tiles: int = 0,
         stages: int = 0, row_groups: int = 0, slices: int = 0, workspace=None, stream=None):
    """Y = fp16(s_a * s1 * (A8 @ W8^.T)); returns y (and the int32 acc if asked)."""
    m = a8.shape[0]
    assert a8.dtype == torch.int8 and a8.is_cuda and a8.stride(1) == 1
    if y is None:
        y = _empty((m, n), torch.float16, a8.device, stream)
    if want_acc and acc is None:
        acc = _empty((m, n), torch.int32, a8.device, stream)
    opts = None
    if variant or k_split or n_tiles or m_tiles or stages or row_groups or slices:
        opts = GemmOpts(variant, k_split, n_tiles, m_tiles, stages, row_groups, slices)
    ws_need = int(lib.w4a8_gemm_workspace_size(m, n, k, g,
                                               ctypes.byref(opts) if opts is not None else None))
    if ws_need and workspace is None:
        workspace = _empty(ws_need, torch.uint8, a8.device, stream, returned=False)
    st = lib.w4a8_gemm(a8.data_ptr(), a8.stride(0), s_a.data_ptr(), m, blob_dev.data_ptr(), n, k,
                       g, y.data_ptr(), y.stride(0),
                       acc.data_ptr() if acc is not None else None,
                       acc.stride(0) if acc is not None else 0,
                       workspace.data_ptr() if workspace is not None else None,
                       workspace.numel() if workspace is not None else 0,
                       ctypes.byref(opts) if opts is not None else None, _stream_of(a8, stream))
    _check(st, "w4a8_gemm")
    return (y, acc) if acc is not None else y


@_on_device
def gemm_noalloc(a8, s_a, blob_dev, n: int, k: int, g: int, y, acc=None, slices: int = 0,
                 stream=None):
    """w4a8_gemm_noalloc: the GEMM with no workspace argument (a K split keeps
    its partial sums in the library's static device scratch).  y (and acc,
    if given) must be preallocated; nothing is allocated here."""
    m = a8.shape[0]
    assert a8.dtype == torch.int8 and a8.is_cuda and a8.stride(1) == 1
    opts = GemmOpts(0, 0, 0, 0, 0, 0, slices) if slices else None
    st = lib.w4a8_gemm_noalloc(a8.data_ptr(), a8.stride(0), s_a.data_ptr(), m,
                               blob_dev.data_ptr(), n, k, g, y.data_ptr(), y.stride(0),
                               acc.data_ptr() if acc is not None else None,
                               acc.stride(0) if acc is not None else 0,
                               ctypes.byref(opts) if opts is not None else None,
                               _stream_of(a8, stream))
    _check(st, "w4a8_gemm_noalloc")
    return (y, acc) if acc is not None else y


@_on_device
def linear(a, blob_dev, n: int, k: int, g: int, y=None, a8=None, s_a=None, acc=None,
           want_acc=False, variant: int = 0, k_split: int = 0, n_tiles: int = 0,
           m_tiles: int = 0, stages: int = 0, row_groups: int = 0, slices: int = 0,
           workgroups: int = 0, workspace=None, stream=None):
    """The whole layer from fp16 activations (fused for small M); returns
    (y, a8, s_a) or (y, a8, s_a, acc)."""
    assert a.dtype == torch.float16 and a.is_cuda and a.dim() == 2 and a.stride(1) == 1
    m = a.shape[0]
    if y is None:
        y = _empty((m, n), torch.float16, a.device, stream)
    if a8 is None:
        a8 = _empty((m, k), torch.int8, a.device, stream)
    if s_a is None:
        s_a = _empty((m,), torch.float16, a.device, stream)
    if want_acc and acc is None:
        acc = _empty((m, n), torch.int32, a.device, stream)
    opts = None
    if variant or k_split or n_tiles or m_tiles or stages or row_groups or slices or workgroups:
        opts = GemmOpts(variant, k_split, n_tiles, m_tiles, stages, row_groups, slices, workgroups)
    ws_opts = opts if (opts is None or variant != 3) else None
    ws_need = 0 if variant == 3 else int(lib.w4a8_gemm_workspace_size(
        m, n, k, g, ctypes.byref(ws_opts) if ws_opts is not None else None))
    if ws_need and workspace is None:
        workspace = _empty(ws_need, torch.uint8, a.device, stream, returned=False)
    st = lib.w4a8_linear(a.data_ptr(), a.stride(0), m, k, blob_dev.data_ptr(), n, g,
                         y.data_ptr(), y.stride(0), a8.data_ptr(), a8.stride(0), s_a.data_ptr(),
                         acc.data_ptr() if acc is not None else None,
                         acc.stride(0) if acc is not None else 0,
                         workspace.data_ptr() if workspace is not None else None,
                         workspace.numel() if workspace is not None else 0,
                         ctypes.byref(opts) if opts is not None else None, _stream_of(a, stream))
    _check(st, "w4a8_linear")
    return (y, a8, s_a, acc) if acc is not None else (y, a8, s_a)


@_on_device
def w4a16(a, blob_dev, n: int, k: int, g: int, y=None, variant: int = 0, k_split: int = 0,
          n_tiles: int = 0, stream=None):
    """W4A16 comparison GEMM on the same blob: fp16 A times fp16-decoded weights."""
    assert a.dtype == torch.float16 and a.is_cuda and a.dim() == 2 and a.stride(1) == 1
    m = a.shape[0]
    if y is None:
        y = _empty((m, n), torch.float16, a.device, stream)
    opts = None
    if variant or k_split or n_tiles:
        opts = GemmOpts(variant, k_split, n_tiles)
    _check(lib.w4a16_gemm(a.data_ptr(), a.stride(0), m, k, blob_dev.data_ptr(), n, g,
                          y.data_ptr(), y.stride(0),
                          ctypes.byref(opts) if opts is not None else None, _stream_of(a, stream)),
           "w4a16_gemm")
    return y


def _elsewhere(name, t, dev):
    return ValueError(f"{name}: expected a CUDA tensor on device {dev}, got one on {t.device}")


def _rows(name, t, dtype, dev, m=None, k=None):
    """Check a 2-D tensor on CUDA device `dev` whose rows are contiguous."""
    if t.dtype is not dtype or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name}: expected a 2-D {dtype} CUDA tensor with contiguous rows")
    if t.get_device() != dev or dev < 0:
        raise _elsewhere(name, t, dev)
    if m is not None and t.shape != (m, k):
        raise ValueError(f"{name}: expected shape ({m}, {k}), got {tuple(t.shape)}")


def _vector(name, t, dtype, dev, n):
    """Check a contiguous tensor of n values on CUDA device `dev`."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} CUDA tensor of {n} values")
    if t.get_device() != dev:
        raise _elsewhere(name, t, dev)


def _int8_out(m, k, a8, s_a, like, stream):
    """The outputs of a per-token quantizer, allocated where not given."""
    if a8 is not None:
        _rows("a8", a8, torch.int8, like.get_device(), m, k)
    if s_a is not None:
        _vector("s_a", s_a, torch.float16, like.get_device(), m)
    if a8 is None:
        a8 = _empty((m, k), torch.int8, like.device, stream)
    if s_a is None:
        s_a = _empty((m,), torch.float16, like.device, stream)
    return a8, s_a


INT_MAX = 2 ** 31 - 1


def _int(name, v):
    """v as the C interface's int: ctypes would pass its low 32 bits."""
    if not 0 <= v <= INT_MAX:
        raise ValueError(f"{name}: {v} is not in 0 .. {INT_MAX}")
    return v


def _bounds(*values):
    """A bound or a window beyond any sequence is none; one below 0 is refused by
    the library."""
    if max(values) > INT_MAX or min(values) < 0:
        return tuple(max(-1, min(v, INT_MAX)) for v in values)
    return values


def _ld(t):
    """Row stride of a 2-D tensor (a single row's stride says nothing)."""
    m, k = t.shape
    ld = t.stride(0) if m > 1 else max(t.stride(0), k)
    return ld if ld <= INT_MAX and m <= INT_MAX else _int("rows or row stride", max(ld, m))


@_on_device
def rms_norm_quant(x, weight, eps: float = 1e-5, residual=None, h=None, a8=None, s_a=None,
                   stream=None):
    """h = x + residual, then the RMS norm of h quantized per token: returns
    (h, a8, s_a), a8 and s_a ready for gemm().  Without a residual h is x.
    h may be given, also as x or residual themselves (in place)."""
    dev = x.get_device()
    _rows("x", x, torch.float16, dev)
    m, k = x.shape
    _vector("weight", weight, torch.float16, dev, k)
    if residual is not None:
        _rows("residual", residual, torch.float16, dev, m, k)
    if h is not None:
        _rows("h", h, torch.float16, dev, m, k)
    elif residual is not None:
        h = _empty((m, k), torch.float16, x.device, stream)
    a8, s_a = _int8_out(m, k, a8, s_a, x, stream)
    _check(lib.w4a8_rms_norm_quant(
        x.data_ptr(), _ld(x), residual.data_ptr() if residual is not None else None,
        _ld(residual) if residual is not None else 0, weight.data_ptr(), eps, m, k,
        h.data_ptr() if h is not None else None, _ld(h) if h is not None else 0,
        a8.data_ptr(), _ld(a8), s_a.data_ptr(), _stream_of(x, stream)), "w4a8_rms_norm_quant")
    return (h if h is not None else x), a8, s_a


@_on_device
def silu_mul_quant(gate, up=None, a8=None, s_a=None, stream=None):
    """silu(gate) * up quantized per token: returns (a8, s_a).  With gate alone,
    its left half is the gate and its right half up (one gate-and-up output)."""
    _rows("gate", gate, torch.float16, gate.get_device())
    if up is None:
        if gate.shape[1] % 2:
            raise ValueError("gate: expected an even number of columns (gate and up side by side)")
        m, k = gate.shape[0], gate.shape[1] // 2
        up_ptr, ldu = gate.data_ptr() + 2 * k, _ld(gate)
    else:
        m, k = gate.shape
        _rows("up", up, torch.float16, gate.get_device(), m, k)
        up_ptr, ldu = up.data_ptr(), _ld(up)
    a8, s_a = _int8_out(m, k, a8, s_a, gate, stream)
    _check(lib.w4a8_silu_mul_quant(gate.data_ptr(), _ld(gate), up_ptr, ldu, m, k, a8.data_ptr(),
                                   _ld(a8), s_a.data_ptr(), _stream_of(gate, stream)),
           "w4a8_silu_mul_quant")
    return a8, s_a


def kv_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda"):
    """A paged int8 KV cache: (cache int8 [num_pages, 2, kv_heads, page_size,
    head_dim], scale float16 [num_pages, 2, kv_heads]), [:, 0] the keys."""
    return (torch.zeros((num_pages, 2, kv_heads, page_size, head_dim), dtype=torch.int8, device=device),
            torch.zeros((num_pages, 2, kv_heads), dtype=torch.float16, device=device))


def rope_table(max_pos: int, rotary_dim: int, base: float = 10000.0, scaling: str | None = None,
               factor: float = 1.0, original_max_pos: int = 8192, low: float = 1.0,
               high: float = 4.0, device="cuda"):
    """cos_sin for rope_append(): float32 [max_pos, rotary_dim], cosines then
    sines, computed in 64 bits from the frequencies base^(-2i / rotary_dim).

    scaling  None
             "linear": every frequency / factor
             "base":   base * factor^(rotary_dim / (rotary_dim - 2)), which
                       leaves the highest frequency and divides the lowest by
                       factor
             "bands":  by the turns within original_max_pos: frequencies of
                       fewer than `low` divided by factor, those of more than
                       `high` kept, a linear blend between (the scheme of
                       Llama-3.1's checkpoints)
    """
    if max_pos < 1 or rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rope_table: max_pos >= 1 and an even rotary_dim >= 2 are needed")
    if factor <= 0 or base <= 0 or (scaling == "bands" and not 0 < low < high):
        raise ValueError("rope_table: factor and base must be positive, and 0 < low < high")
    exponent = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = base ** -exponent
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "bands":
        turns = original_max_pos * freq / (2 * np.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
    elif scaling not in (None, "base"):
        raise ValueError(f"rope_table: unknown scaling {scaling!r}")
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().to(device)


def _cache(cache, scale, dev):
    """Check a paged cache on CUDA device `dev`; returns (pages, heads, page
    size, head dim)."""
    if cache.dtype is not torch.int8 or cache.dim() != 5 or cache.shape[1] != 2:
        raise ValueError("cache: expected an int8 CUDA tensor [pages, 2, kv_heads, page_size, head_dim]")
    pages, _, heads, page, dim = cache.shape
    if cache.stride()[1:] != (heads * page * dim, page * dim, dim, 1):
        raise ValueError("cache: the values of a page must be contiguous")
    if scale.dtype is not torch.float16 or scale.shape != (pages, 2, heads) \
            or scale.stride()[1:] != (heads, 1):
        raise ValueError(f"scale: expected a float16 CUDA tensor [{pages}, 2, {heads}], "
                         "contiguous within a page")
    if cache.get_device() != dev:
        raise _elsewhere("cache", cache, dev)
    if scale.get_device() != dev:
        raise _elsewhere("scale", scale, dev)
    return pages, heads, page, dim


def _kv_view(cache, scale, block_table, seq_lens, cu_q, q):
    """The C view of a cache and a batch for the new tokens of q, its tensors
    checked."""
    total_q, dev = q.shape[0], q.get_device()
    pages, heads, page, dim = _cache(cache, scale, dev)
    if block_table.dtype is not torch.int32 or block_table.dim() != 2 \
            or (block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("block_table: expected an int32 CUDA tensor [batch, pages of a sequence]")
    if block_table.get_device() != dev:
        raise _elsewhere("block_table", block_table, dev)
    batch, max_pages = block_table.shape
    _vector("seq_lens", seq_lens, torch.int32, dev, batch)
    if cu_q is not None:
        _vector("cu_q", cu_q, torch.int32, dev, batch + 1)
    elif total_q != batch:
        raise ValueError(f"without cu_q each of the {batch} sequences brings one token, got {total_q}")
    table_ld = block_table.stride(0) if batch > 1 else max(block_table.stride(0), max_pages)
    if table_ld > INT_MAX or batch > INT_MAX or pages > INT_MAX:
        _int("pages, sequences or the block table's row stride", max(table_ld, batch, pages))
    return KvView(cache.data_ptr(), scale.data_ptr(),
                  cache.stride(0) if pages > 1 else 2 * heads * page * dim,
                  scale.stride(0) if pages > 1 else 2 * heads, pages, page, heads, dim,
                  block_table.data_ptr(), table_ld, max_pages, seq_lens.data_ptr(),
                  cu_q.data_ptr() if cu_q is not None else None, batch, total_q)


def _heads(name, t, dev, tokens=None, heads=None, dim=None):
    """Check a [tokens, heads, dim] float16 tensor on CUDA device `dev` whose rows
    (all heads of a token) are contiguous; returns the row stride."""
    if t.dtype is not torch.float16 or t.dim() != 3:
        raise ValueError(f"{name}: expected a float16 CUDA tensor [tokens, heads, head_dim]")
    if t.get_device() != dev or dev < 0:
        raise _elsewhere(name, t, dev)
    n, h, d = t.shape
    if (tokens is not None and n != tokens) or (heads is not None and h != heads) \
            or (dim is not None and d != dim):
        raise ValueError(f"{name}: expected shape ({tokens}, {heads or 'heads'}, {dim}), got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (h > 1 and s[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    ld = s[0] if n > 1 else max(s[0], h * d)
    return ld if ld <= INT_MAX and n <= INT_MAX else _int(f"{name}: tokens or row stride", max(ld, n))


@_on_device
def rope_append(q, k, v, cos_sin, cache, scale, block_table, seq_lens, cu_q=None,
                interleaved: bool = False, out=None, stream=None, positions=None):
    """Rotate q [tokens, heads, dim] and k by position and append k and v
    [tokens, kv_heads, dim] to the paged cache; returns the rotated q (a new
    tensor, or `out`, which may be q).  cos_sin [max_pos, rotary_dim] is
    rope_table()'s, or None for no rotation.  positions, int32 [tokens], are the
    angles' where they differ from the tokens' places in the cache (drafted
    trees).  See w4a8_rope_append."""
    dev = q.get_device()
    tokens, heads, dim = q.shape
    view = _kv_view(cache, scale, block_table, seq_lens, cu_q, q)
    ldq = _heads("q", q, dev, tokens, None, view.head_dim)
    ldk = _heads("k", k, dev, tokens, view.kv_heads, view.head_dim)
    ldv = _heads("v", v, dev, tokens, view.kv_heads, view.head_dim)
    rotary = max_pos = 0
    if cos_sin is not None:
        if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin: expected a contiguous float32 CUDA tensor [max_pos, rotary_dim]")
        if cos_sin.get_device() != dev:
            raise _elsewhere("cos_sin", cos_sin, dev)
        max_pos, rotary = cos_sin.shape
        _int("cos_sin: positions or rotary_dim", max(max_pos, rotary))
    if out is None:
        out, ldo = _empty((tokens, heads, dim), torch.float16, q.device, stream), heads * dim
    else:
        ldo = _heads("out", out, dev, tokens, heads, dim)
    if positions is not None:
        _vector("positions", positions, torch.int32, dev, tokens)
        _check(lib.w4a8_rope_append_at(
            q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, heads,
            cos_sin.data_ptr() if cos_sin is not None else None, rotary, max_pos, int(interleaved),
            positions.data_ptr(), ctypes.byref(view), out.data_ptr(), ldo, _stream_of(q, stream)),
            "w4a8_rope_append_at")
        return out
    _check(lib.w4a8_rope_append(
        q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, heads,
        cos_sin.data_ptr() if cos_sin is not None else None, rotary, max_pos, int(interleaved),
        ctypes.byref(view), out.data_ptr(), ldo, _stream_of(q, stream)), "w4a8_rope_append")
    return out


@_on_device
def paged_attention(q, cache, scale_kv, block_table, seq_lens, cu_q=None, max_q: int | None = None,
                    max_len: int | None = None, scale: float | None = None, window: int = 0, out=None, workspace=None,
                    stream=None):
    """Causal attention of q [tokens, heads, dim] over the paged int8 cache;
    returns o like q.  max_q and max_len bound the new tokens of a sequence
    and seq_lens on the host (defaults: all of q, and what the block table
    holds); scale defaults to dim ** -0.5.  See w4a8_paged_attention."""
    dev = q.get_device()
    tokens, heads, dim = q.shape
    view = _kv_view(cache, scale_kv, block_table, seq_lens, cu_q, q)
    ldq = _heads("q", q, dev, tokens, None, view.head_dim)
    if out is None:
        out, ldo = _empty((tokens, heads, dim), torch.float16, q.device, stream), heads * dim
    else:
        ldo = _heads("out", out, dev, tokens, heads, dim)
    if max_len is None:
        max_len = view.max_pages * view.page_size
    if max_q is None:
        max_q = 1 if cu_q is None else tokens
    max_q, max_len, window = _bounds(max_q, max_len, window)
    need = lib.w4a8_paged_attention_workspace_size(ctypes.byref(view), heads, max_q, max_len)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream, returned=False)
    elif workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace: expected a contiguous CUDA tensor on device {dev}")
    _check(lib.w4a8_paged_attention(
        q.data_ptr(), ldq, heads, ctypes.byref(view), max_q, max_len,
        dim ** -0.5 if scale is None else scale, window, out.data_ptr(), ldo,
        workspace.data_ptr() if workspace is not None else None,
        workspace.numel() * workspace.element_size() if workspace is not None else 0,
        _stream_of(q, stream)), "w4a8_paged_attention")
    return out


def _tree(parents, seq_lens, cu_q, dev):
    """Check a batch of drafted tokens; returns (tokens, batch)."""
    tokens = parents.shape[0] if parents.dim() == 1 else -1
    _vector("parents", parents, torch.int32, dev, tokens)
    batch = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    _vector("seq_lens", seq_lens, torch.int32, dev, batch)
    if cu_q is not None:
        _vector("cu_q", cu_q, torch.int32, dev, batch + 1)
    elif tokens != batch:
        raise ValueError(f"without cu_q each of the {batch} sequences has one node, got {tokens}")
    if max(tokens, batch) > INT_MAX:
        _int("nodes or sequences", max(tokens, batch))
    return tokens, batch


def _most_nodes(tokens, cu_q, max_q):
    return 1 if cu_q is None else tokens if max_q is None else min(max_q, tokens)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _mask(mask, dev, tokens):
    if mask.dtype is not torch.int32 or mask.dim() != 2 or mask.shape[0] != tokens or mask.shape[1] < 1 \
            or (mask.stride(1) != 1 and mask.shape[1] > 1):
        raise ValueError(f"mask: expected an int32 CUDA tensor [{tokens}, words] with contiguous rows")
    if mask.get_device() != dev or dev < 0:
        raise _elsewhere("mask", mask, dev)
    return _ld(mask)


@_on_device
def tree_mask(parents, seq_lens, cu_q=None, max_q: int | None = None, mask=None, positions=None, stream=None):
    """(mask int32 [tokens, ceil(max_q / 32)], positions int32 [tokens]) of
    drafted trees: parents int32 [tokens] holds each node's parent within its
    sequence, -1 for none.  max_q bounds the nodes of a sequence (default: all
    of them).  See w4a8_tree_mask."""
    dev = parents.get_device()
    tokens, batch = _tree(parents, seq_lens, cu_q, dev)
    if mask is not None:
        ld = _mask(mask, dev, tokens)
    if positions is not None:
        _vector("positions", positions, torch.int32, dev, tokens)
    if mask is None:
        words = max(1, -(-_most_nodes(tokens, cu_q, max_q) // 32))
        mask, ld = _empty((tokens, words), torch.int32, parents.device, stream), words
    if positions is None:
        positions = _empty((tokens,), torch.int32, parents.device, stream)
    _check(lib.w4a8_tree_mask(parents.data_ptr(), seq_lens.data_ptr(), _ptr(cu_q), batch, tokens, mask.data_ptr(),
                              ld, mask.shape[1], positions.data_ptr(), _stream_of(parents, stream)),
           "w4a8_tree_mask")
    return mask, positions


@_on_device
def tree_attention(q, cache, scale_kv, block_table, seq_lens, mask, cu_q=None, max_q: int | None = None,
                   max_len: int | None = None, scale: float | None = None, window: int = 0, out=None,
                   workspace=None, stream=None):
    """Attention of drafted tokens q [tokens, heads, dim] over the paged int8
    cache, which holds them already: all positions before the sequence's drafted
    tokens, and of these the ones that mask (tree_mask()'s) names.  Other
    arguments as paged_attention's.  See w4a8_tree_attention."""
    dev = q.get_device()
    tokens, heads, dim = q.shape
    view = _kv_view(cache, scale_kv, block_table, seq_lens, cu_q, q)
    ldq = _heads("q", q, dev, tokens, None, view.head_dim)
    ld_mask = _mask(mask, dev, tokens)
    if out is None:
        out, ldo = _empty((tokens, heads, dim), torch.float16, q.device, stream), heads * dim
    else:
        ldo = _heads("out", out, dev, tokens, heads, dim)
    if max_len is None:
        max_len = view.max_pages * view.page_size
    if max_q is None:
        max_q = 1 if cu_q is None else tokens
    max_q, max_len, window = _bounds(max_q, max_len, window)
    need = lib.w4a8_tree_attention_workspace_size(ctypes.byref(view), heads, max_q, max_len)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, q.device, stream, returned=False)
    elif workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace: expected a contiguous CUDA tensor on device {dev}")
    _check(lib.w4a8_tree_attention(
        q.data_ptr(), ldq, heads, ctypes.byref(view), mask.data_ptr(), ld_mask, mask.shape[1], max_q, max_len,
        dim ** -0.5 if scale is None else scale, window, out.data_ptr(), ldo, _ptr(workspace),
        workspace.numel() * workspace.element_size() if workspace is not None else 0,
        _stream_of(q, stream)), "w4a8_tree_attention")
    return out


@_on_device
def tree_accept(drafted, parents, sampled, seq_lens, cu_q=None, max_q: int | None = None, stream=None):
    """The nodes of drafted trees that sampled tokens confirm, all int32: (path
    [batch, max_q] nodes in order, then -1, count [batch], tokens [batch] drawn
    after the last of them, seq_lens [batch] without the others).  max_q bounds the
    nodes of a path (default: all of them).  See w4a8_tree_accept."""
    dev = drafted.get_device()
    if dev < 0:
        raise _elsewhere("drafted", drafted, dev)
    tokens, batch = _tree(parents, seq_lens, cu_q, dev)
    _vector("drafted", drafted, torch.int32, dev, tokens)
    _vector("sampled", sampled, torch.int32, dev, tokens)
    most = max(1, _most_nodes(tokens, cu_q, max_q))
    new = lambda *shape: _empty(shape, torch.int32, drafted.device, stream)
    path, count, following, lens = new(batch, most), new(batch), new(batch), new(batch)
    _check(lib.w4a8_tree_accept(drafted.data_ptr(), parents.data_ptr(), sampled.data_ptr(), seq_lens.data_ptr(),
                                _ptr(cu_q), batch, tokens, path.data_ptr(), most, most, count.data_ptr(),
                                following.data_ptr(), lens.data_ptr(), _stream_of(drafted, stream)),
           "w4a8_tree_accept")
    return path, count, following, lens


@_on_device
def kv_keep(cache, scale, block_table, seq_lens, path, count, cu_q=None, stream=None):
    """Keys and values of confirmed nodes (tree_accept()'s path and count) moved
    to the places behind their sequence's certain tokens, in place; seq_lens and
    cu_q are those that the nodes were appended with.  See w4a8_kv_keep."""
    dev = cache.get_device()
    if dev < 0:
        raise _elsewhere("cache", cache, dev)
    view = _kv_view(cache, scale, block_table, seq_lens, cu_q, path)
    batch = view.batch
    if path.dtype is not torch.int32 or path.dim() != 2 or path.shape[0] != batch or path.shape[1] < 1 \
            or (path.stride(1) != 1 and path.shape[1] > 1):
        raise ValueError(f"path: expected an int32 CUDA tensor [{batch}, nodes] with contiguous rows")
    if path.get_device() != dev:
        raise _elsewhere("path", path, dev)
    _vector("count", count, torch.int32, dev, batch)
    if cu_q is not None:
        view.total_q = M_MAX             # not known here, and only a bound
    _check(lib.w4a8_kv_keep(ctypes.byref(view), path.data_ptr(), _ld(path), path.shape[1], count.data_ptr(),
                            _stream_of(cache, stream)), "w4a8_kv_keep")


@_on_device
def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, probs=None, workspace=None,
           stream=None):
    """A token for each row of logits [rows, vocab] (float16 or float32) from the
    random numbers u, float32 [rows] in [0, 1): returns (tokens int32 [rows], probs
    float32 [rows], the share of the kept weights that each token has).  Settings
    are numbers, or CUDA tensors of one value a row (float32, top_k int32);
    temperature 0 takes the largest logit.  See w4a8_sample."""
    dev = logits.get_device()
    f32 = logits.dtype is torch.float32
    _rows("logits", logits, torch.float32 if f32 else torch.float16, dev)
    rows, vocab = logits.shape
    _vector("u", u, torch.float32, dev, rows)
    s = Sampling()
    for name, value, kind in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                              ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if isinstance(value, torch.Tensor):
            _vector(name, value, kind, dev, rows)
            setattr(s, name + "_dev", value.data_ptr())
        elif kind is torch.int32:
            s.top_k = max(0, min(value, INT_MAX))
        else:
            setattr(s, name, value)
    if tokens is None:
        tokens = _empty((rows,), torch.int32, logits.device, stream)
    else:
        _vector("tokens", tokens, torch.int32, dev, rows)
    if probs is None:
        probs = _empty((rows,), torch.float32, logits.device, stream)
    else:
        _vector("probs", probs, torch.float32, dev, rows)
    ld = _ld(logits)
    need = lib.w4a8_sample_workspace_size(int(f32), rows, vocab)
    if need and workspace is None:
        workspace = _empty(need, torch.uint8, logits.device, stream, returned=False)
    elif workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace: expected a contiguous CUDA tensor on device {dev}")
    _check(lib.w4a8_sample(logits.data_ptr(), int(f32), ld, rows, vocab, u.data_ptr(), ctypes.byref(s),
                           tokens.data_ptr(), probs.data_ptr(), _ptr(workspace),
                           workspace.numel() * workspace.element_size() if workspace is not None else 0,
                           _stream_of(logits, stream)), "w4a8_sample")
    return tokens, probs


def _table(block_table, dev):
    if block_table.dtype is not torch.int32 or block_table.dim() != 2 or block_table.shape[1] < 1 \
            or (block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("block_table: expected an int32 CUDA tensor [batch, pages of a sequence]")
    if block_table.get_device() != dev or dev < 0:
        raise _elsewhere("block_table", block_table, dev)
    return (*block_table.shape, _ld(block_table))


def _pool_refs(refs, dev):
    pages = refs.shape[0] if refs.dim() == 1 else -1
    _vector("refs", refs, torch.int32, dev, pages)
    return _int("pages", pages)


@_on_device
def kv_fork(block_table, seq_lens, refs, parent, page_size: int, stream=None):
    """(block_table, seq_lens, refs) in which row i continues sequence parent[i]
    (int32 [rows]; -1: an empty row) and pages without a row are free.  refs,
    int32 [pages], counts how often tables name each page.  The arguments stay as
    they are.  See w4a8_kv_fork."""
    dev = block_table.get_device()
    batch, width, ld = _table(block_table, dev)
    _vector("seq_lens", seq_lens, torch.int32, dev, batch)
    pages = _pool_refs(refs, dev)
    rows = parent.shape[0] if parent.dim() == 1 else -1
    _vector("parent", parent, torch.int32, dev, rows)
    _int("rows", rows)
    _int("page_size", page_size)
    new = lambda *shape: _empty(shape, torch.int32, block_table.device, stream)
    table, lens, counts = new(rows, width), new(rows), new(pages)
    _check(lib.w4a8_kv_fork(block_table.data_ptr(), ld, width, seq_lens.data_ptr(), batch, refs.data_ptr(), pages,
                            page_size, parent.data_ptr(), rows, table.data_ptr(), width, lens.data_ptr(),
                            counts.data_ptr(), _stream_of(block_table, stream)), "w4a8_kv_fork")
    return table, lens, counts


@_on_device
def kv_alloc(block_table, seq_lens, refs, tokens, page_size: int, stream=None):
    """Pages for the next tokens (a number, or int32 [batch]) of each sequence:
    (block_table, seq_lens with them, refs, src, dst, counts).  Pages src[i] are to
    be copied to dst[i], for i < counts[0] (kv_copy_pages()); counts[1] entries got
    no page.  A sequence whose length was lowered gives up shared pages behind its
    tokens before, by a kv_fork() into another row.  The arguments stay as they are.
    See w4a8_kv_alloc."""
    dev = block_table.get_device()
    batch, width, ld = _table(block_table, dev)
    _vector("seq_lens", seq_lens, torch.int32, dev, batch)
    pages = _pool_refs(refs, dev)
    each = isinstance(tokens, torch.Tensor)
    if each:
        _vector("tokens", tokens, torch.int32, dev, batch)
    else:
        _int("tokens", tokens)
    _int("page_size", page_size)
    new = lambda *shape: _empty(shape, torch.int32, block_table.device, stream)
    table, lens, owners, src, dst, counts = new(batch, width), new(batch), new(pages), new(batch), new(batch), new(2)
    need = lib.w4a8_kv_alloc_workspace_size(batch, pages)
    workspace = _empty(need, torch.uint8, block_table.device, stream, returned=False)
    _check(lib.w4a8_kv_alloc(block_table.data_ptr(), ld, width, seq_lens.data_ptr(), batch, refs.data_ptr(), pages,
                             page_size, tokens.data_ptr() if each else None, 0 if each else tokens,
                             table.data_ptr(), width, lens.data_ptr(), owners.data_ptr(), src.data_ptr(),
                             dst.data_ptr(), counts.data_ptr(), workspace.data_ptr(), need,
                             _stream_of(block_table, stream)), "w4a8_kv_alloc")
    return table, lens, owners, src, dst, counts


@_on_device
def kv_compact(block_table, refs, stream=None):
    """The pages in use at the front of the pool: (block_table, refs, place, src,
    dst, counts).  Pages src[i] are to be copied to dst[i], for i < counts[0]
    (kv_copy_pages()); place [pages] says where each page is then.  The arguments
    stay as they are.  See w4a8_kv_compact."""
    dev = block_table.get_device()
    batch, width, ld = _table(block_table, dev)
    pages = _pool_refs(refs, dev)
    new = lambda *shape: _empty(shape, torch.int32, block_table.device, stream)
    moves = pages // 2
    table, owners, place, src, dst, counts = new(batch, width), new(pages), new(pages), new(moves), new(moves), new(2)
    need = lib.w4a8_kv_compact_workspace_size(pages)
    workspace = _empty(need, torch.uint8, block_table.device, stream, returned=False)
    _check(lib.w4a8_kv_compact(block_table.data_ptr(), ld, width, batch, refs.data_ptr(), pages, table.data_ptr(),
                               width, owners.data_ptr(), place.data_ptr(), src.data_ptr(), dst.data_ptr(),
                               counts.data_ptr(), workspace.data_ptr(), need, _stream_of(block_table, stream)),
           "w4a8_kv_compact")
    return table, owners, place, src, dst, counts


@_on_device
def kv_copy_pages(cache, scale, src, dst, count=None, stream=None):
    """Pages src[i] of a cache copied with their scales to dst[i] (int32), in
    place, for all i or those below count[0] (int32, on the device).  See
    w4a8_kv_copy_pages."""
    dev = cache.get_device()
    if dev < 0:
        raise _elsewhere("cache", cache, dev)
    pages, heads, page, dim = _cache(cache, scale, dev)
    pairs = src.shape[0] if src.dim() == 1 else -1
    _vector("src", src, torch.int32, dev, pairs)
    _vector("dst", dst, torch.int32, dev, pairs)
    _int("pairs", pairs)
    if count is not None and (count.dtype is not torch.int32 or count.numel() < 1 or count.get_device() != dev):
        raise ValueError(f"count: expected an int32 CUDA tensor on device {dev}")
    _check(lib.w4a8_kv_copy_pages(
        cache.data_ptr(), scale.data_ptr(), cache.stride(0) if pages > 1 else 2 * heads * page * dim,
        scale.stride(0) if pages > 1 else 2 * heads, pages, page, heads, dim, src.data_ptr(), dst.data_ptr(), pairs,
        _ptr(count), _stream_of(cache, stream)), "w4a8_kv_copy_pages")


@_on_device
def read_probe(buf, offset: int, nbytes: int, workgroups: int, sink, stream=None):
    """Measurement aid: a read-only stream over nbytes of the uint8 CUDA tensor
    `buf` from byte `offset` (w4a8_read_probe); sink is an int32 CUDA tensor of
    at least `workgroups` elements."""
    assert buf.is_cuda and 0 <= offset and offset + nbytes <= buf.numel() * buf.element_size()
    assert sink.numel() >= workgroups
    _check(lib.w4a8_read_probe(buf.data_ptr() + offset, nbytes, workgroups, sink.data_ptr(),
                               _stream_of(buf, stream)), "w4a8_read_probe")
