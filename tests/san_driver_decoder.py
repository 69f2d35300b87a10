"""Driver run in a child process against the host-only sanitized build of the
decoder-layer entry points (see test_decoder_host.py): thousands of random,
extreme argument sets.  Fake pointers are never dereferenced: a call that
passes validation reaches a stub, which aborts if its launch would not fit.

    python san_driver_decoder.py LIB
"""
import ctypes
import json
import sys

import numpy as np


def main():
    L = ctypes.CDLL(sys.argv[1])
    P, I, Z, F, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_longlong

    class View(ctypes.Structure):
        _fields_ = [("data", P), ("scale", P), ("page_stride", LL), ("scale_stride", LL),
                    ("num_pages", I), ("page_size", I), ("kv_heads", I), ("head_dim", I),
                    ("table", P), ("table_ld", I), ("max_pages", I), ("lens", P), ("cu_q", P),
                    ("batch", I), ("total_q", I)]

    L.w4a8_rms_norm_quant.argtypes = [P, I, P, I, P, F, I, I, P, I, P, I, P, P]
    L.w4a8_silu_mul_quant.argtypes = [P, I, P, I, I, I, P, I, P, P]
    L.w4a8_rope_append.argtypes = [P, I, P, I, P, I, I, P, I, I, I, P, P, I, P]
    L.w4a8_paged_attention_workspace_size.argtypes = [P, I, I, I]
    L.w4a8_paged_attention_workspace_size.restype = Z
    L.w4a8_paged_attention.argtypes = [P, I, I, P, I, I, F, I, P, I, P, Z, P]
    rng = np.random.default_rng(3)
    pick = lambda xs: xs[int(rng.integers(len(xs)))]
    ints = [-(2 ** 31), -1, 0, 1, 2, 3, 15, 16, 31, 64, 100, 128, 1000, 4096, 65536, 1 << 20, 1 << 22,
            (1 << 22) + 1, 2 ** 30, 2 ** 31 - 1]
    ptrs = [None, 4096, 4104, 4096, 1 << 40]
    floats = [0.0, 1e-5, 1.0, -1.0, float("inf"), float("nan"), 3e38]
    seen = {}
    for it in range(20000):
        sane = rng.random() < 0.7
        page, heads, dim = pick([16, 32, 64, 256, 1024]), pick([1, 2, 8, 64]), 16 * int(rng.integers(1, 17))
        batch = pick([0, 1, 3, 64, 4096, 1 << 20, 1 << 22])
        v = View(4096, 4096, 2 * heads * page * dim, 2 * heads, pick([1, 7, 1 << 20]), page, heads, dim,
                 4096, 64, pick([1, 64]), 4096, None, batch, batch)
        if rng.random() < 0.6:
            v.cu_q, v.total_q = 4096, pick([1, 17, 5000, 1 << 18, 1 << 22])
        if not sane:
            for _ in range(int(rng.integers(1, 4))):
                name, kind = pick(View._fields_)
                setattr(v, name, pick(ptrs) if kind is P else pick(ints))
        q_heads = heads * pick([1, 2, 4, 7, 64]) if sane else pick(ints)
        ld = 4096 * 256 if rng.random() < 0.8 else pick(ints)
        vp = ctypes.byref(v) if rng.random() < 0.98 else None
        a, b, c, d = (pick(ptrs) if rng.random() < 0.2 else 4096 for _ in range(4))
        max_q, max_len = pick(ints), pick(ints)
        rotary = pick([0, 16, dim, dim // 2, -16, 272, 8])
        need = L.w4a8_paged_attention_workspace_size(vp, q_heads, max_q, max_len)
        ws = need if rng.random() < 0.8 else pick([0, 16, 1 << 20])
        out = {
            "append": L.w4a8_rope_append(a, ld, b, ld, c, ld, q_heads, d, rotary, pick(ints), 1, vp, a, ld, None),
            "attention": L.w4a8_paged_attention(a, ld, q_heads, vp, max_q, max_len, pick(floats),
                                                pick([0, 0, 5, -1]), b, ld, c, ws, None),
            "norm": L.w4a8_rms_norm_quant(a, pick(ints), pick(ptrs), pick(ints), b, pick(floats), pick(ints),
                                          pick(ints), pick(ptrs), pick(ints), c, pick(ints), d, None),
            "swiglu": L.w4a8_silu_mul_quant(a, pick(ints), b, pick(ints), pick(ints), pick(ints), c,
                                            pick(ints), d, None),
        }
        for name, status in out.items():
            assert 0 <= status <= 7, (name, status)
            seen.setdefault(name, set()).add(status)
    print(json.dumps({k: sorted(v) for k, v in seen.items()}))


if __name__ == "__main__":
    main()
