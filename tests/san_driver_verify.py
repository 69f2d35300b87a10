"""Driver run in a child process against the host-only sanitized build of
verify_api.cpp (see test_verify_host.py): thousands of random, extreme argument
sets.  Fake pointers are never dereferenced: a call that passes validation
reaches a stub, which aborts if its launch would not fit.

    python san_driver_verify.py LIB
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

    class Sampling(ctypes.Structure):
        _fields_ = [("temperature", F), ("top_k", I), ("top_p", F), ("min_p", F), ("temperature_dev", P),
                    ("top_k_dev", P), ("top_p_dev", P), ("min_p_dev", P)]

    L.w4a8_tree_mask.argtypes = [P, P, P, I, I, P, I, I, P, P]
    L.w4a8_tree_attention_workspace_size.argtypes = [P, I, I, I]
    L.w4a8_tree_attention_workspace_size.restype = Z
    L.w4a8_tree_attention.argtypes = [P, I, I, P, P, I, I, I, I, F, I, P, I, P, Z, P]
    L.w4a8_tree_accept.argtypes = [P, P, P, P, P, I, I, P, I, I, P, P, P, P]
    L.w4a8_kv_keep.argtypes = [P, P, I, I, P, P]
    L.w4a8_sample_workspace_size.argtypes, L.w4a8_sample_workspace_size.restype = [I, I, I], Z
    L.w4a8_sample.argtypes = [P, I, I, I, I, P, P, P, P, P, Z, P]
    L.w4a8_kv_fork.argtypes = [P, I, I, P, I, P, I, I, P, I, P, I, P, P, P]
    L.w4a8_kv_alloc_workspace_size.argtypes, L.w4a8_kv_alloc_workspace_size.restype = [I, I], Z
    L.w4a8_kv_alloc.argtypes = [P, I, I, P, I, P, I, I, P, I, P, I, P, P, P, P, P, P, Z, P]
    L.w4a8_kv_compact_workspace_size.argtypes, L.w4a8_kv_compact_workspace_size.restype = [I], Z
    L.w4a8_kv_compact.argtypes = [P, I, I, I, P, I, P, I, P, P, P, P, P, P, Z, P]
    L.w4a8_kv_copy_pages.argtypes = [P, P, LL, LL, I, I, I, I, P, P, I, P, P]
    rng = np.random.default_rng(4)
    pick = lambda xs: xs[int(rng.integers(len(xs)))]
    ints = [-(2 ** 31), -1, 0, 1, 2, 3, 15, 16, 31, 64, 100, 128, 1000, 4096, 65536, 1 << 20, 1 << 22,
            (1 << 22) + 1, 2 ** 30, 2 ** 31 - 1]
    ptrs = [None, 4096, 4104, 4097, 1 << 40]
    floats = [0.0, 1e-5, 1.0, -1.0, float("inf"), float("nan"), 3e38]
    seen = {}
    for it in range(20000):
        odd = rng.random() < 0.3
        some = lambda value: pick(ints) if odd and rng.random() < 0.3 else value
        at = lambda value=8192: pick(ptrs) if odd and rng.random() < 0.2 else value
        page, heads, dim = pick([16, 32, 64, 256, 1024]), pick([1, 2, 8, 64, 4096]), 16 * int(rng.integers(1, 17))
        batch = pick([0, 1, 3, 64, 4096, 1 << 20, 1 << 22])
        pages = pick([1, 7, 1 << 20, 1 << 22])
        v = View(4096, 4096, 2 * heads * page * dim, 2 * heads, pages, page, heads, dim,
                 4096, 64, pick([1, 64]), 4096, None, batch, batch)
        total = batch
        if rng.random() < 0.6:
            total = pick([0, 1, 17, 5000, 1 << 18, 1 << 22])
            v.cu_q, v.total_q = 4096, total
        cu = v.cu_q
        if odd:
            for _ in range(int(rng.integers(0, 3))):
                name, kind = pick(View._fields_)
                setattr(v, name, pick(ptrs) if kind is P else pick(ints))
        q_heads = some(heads * pick([1, 2, 4, 7, 64]))
        vp = ctypes.byref(v) if rng.random() < 0.98 else None
        max_q, max_len = pick(ints), pick(ints)
        need = L.w4a8_tree_attention_workspace_size(vp, q_heads, max_q, max_len)
        ws = need if rng.random() < 0.8 else pick([0, 16, 1 << 20])
        words, ld = some(pick([1, 2, 40])), some(64)
        s = Sampling(pick(floats) if odd else 0.7, pick(ints), pick(floats), pick(floats) if odd else 0.0,
                     at(None), at(None), at(None), at(None))
        sp = ctypes.byref(s) if rng.random() < 0.98 else None
        b, t, width, n = some(batch), some(total), some(pick([1, 64, 2000])), some(pages)
        size = some(page)
        a_need = L.w4a8_kv_alloc_workspace_size(b, n) if rng.random() < 0.9 else 16
        c_need = L.w4a8_kv_compact_workspace_size(n) if rng.random() < 0.9 else 0
        f32, vocab = pick([0, 1]), some(pick([1, 50257, 1 << 19]))
        s_need = L.w4a8_sample_workspace_size(f32, b, vocab) if rng.random() < 0.9 else 64
        out = {
            "mask": L.w4a8_tree_mask(at(), at(), at(cu), b, t, at(), ld, words, at(), None),
            "attention": L.w4a8_tree_attention(at(), some(4096 * 256), q_heads, vp, at(), ld, words, max_q, max_len,
                                               pick(floats), pick([0, 0, 5, -1]), at(), some(4096 * 256), at(), ws, None),
            "accept": L.w4a8_tree_accept(at(), at(), at(), at(), at(cu), b, t, at(), ld, words, at(), at(), at(), None),
            "keep": L.w4a8_kv_keep(vp, at(), ld, words, at(), None),
            "sample": L.w4a8_sample(at(), f32, some(1 << 19), b, vocab, at(), sp, at(), at(), at(), s_need, None),
            "fork": L.w4a8_kv_fork(at(), some(2000), width, at(), b, at(), n, size, at(), some(pick([0, 5, 1 << 20])),
                                   at(12288), some(2000), at(12288), at(12288), None),
            "alloc": L.w4a8_kv_alloc(at(), some(2000), width, at(), b, at(), n, size, at(), some(3), at(12288), some(2000),
                                     at(12288), at(12288), at(), at(), at(), at(), a_need, None),
            "compact": L.w4a8_kv_compact(at(), some(2000), width, b, at(), n, at(12288), some(2000), at(12288), at(), at(),
                                         at(), at(), at(), c_need, None),
            "copy": L.w4a8_kv_copy_pages(at(), at(), v.page_stride, v.scale_stride, n, size, some(heads), some(dim), at(),
                                         at(), b, at(), None),
        }
        for name, status in out.items():
            assert 0 <= status <= 7, (name, status)
            seen.setdefault(name, set()).add(status)
    print(json.dumps({k: sorted(v) for k, v in seen.items()}))


if __name__ == "__main__":
    main()
