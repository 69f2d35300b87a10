"""Plain numpy implementations, in 64 bits, of the decoder-layer operators:
the yardstick of their GPU tests.  Values before quantization are returned
unrounded; the tests derive what the int8 codes may differ by."""
import numpy as np


def rms_norm(x, residual, weight, eps):
    """(h float16, y float64) of fp16 inputs; h is x without a residual."""
    h = x if residual is None else (x.astype(np.float64) + residual.astype(np.float64)).astype(np.float16)
    h64 = h.astype(np.float64)
    mean = (h64 * h64).mean(axis=1, keepdims=True)
    return h, h64 / np.sqrt(mean + eps) * weight.astype(np.float64)


def silu_mul(gate, up):
    g = gate.astype(np.float64)
    return g / (1.0 + np.exp(-g)) * up.astype(np.float64)


def half_ulp16(v):
    """Half the spacing of float16 at |v| (subnormal spacing below 2^-14)."""
    v = np.maximum(np.abs(np.asarray(v, dtype=np.float64)), 2.0 ** -14)
    return 2.0 ** (np.floor(np.log2(v)) - 11)


# What fp32 arithmetic may add to a value computed by a few rounded operations
# from sums of positive terms: a dozen roundings of 2^-24 each.
FP32 = 12 * 2.0 ** -24


def check_int8_rows(a8, s_a, y, rel=FP32):
    """a8 * s_a stands for y: every scale is the fp16 nearest to amax / 127
    (up to fp32 error of amax before that rounding), every code the integer
    nearest to y / s_a, up to the same error of y and of the reciprocal."""
    amax = np.abs(y).max(axis=1)
    want = amax / 127.0
    s = s_a.astype(np.float64)
    assert (np.abs(s - want) <= half_ulp16(want) + rel * want).all()
    zero = s == 0
    assert (a8[zero] == 0).all()
    q = y[~zero] / s[~zero, None]
    q = np.clip(q, -127, 127)          # a subnormal scale may round down far
    # 3 more roundings: the reciprocal, the product with it, the scaled value
    assert (np.abs(a8[~zero] - q) <= 0.5 + 127.5 * (rel + 3 * 2.0 ** -24)).all()


def rotate(x, pos, cos_sin, interleaved):
    """x [heads, dim] of one token at position pos, in float64."""
    out = x.astype(np.float64).copy()
    half = cos_sin.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(cos_sin[pos, i]), float(cos_sin[pos, i + half])
        va, vb = out[:, a].copy(), out[:, b].copy()
        out[:, a] = va * c - vb * s
        out[:, b] = vb * c + va * s
    return out


def attention(q, cache, scale_kv, table, lens, cu, scale, window=0):
    """(o, bound) [tokens, heads, dim] float64 over a paged int8 cache, row by
    row; a row that sees no key is 0, pages outside the pool are not seen.

    bound is what the kernels' arithmetic may add to o: half an fp16 ulp of
    the result; softmax weights rounded to fp16 (2^-11 of each, so of
    sum p |v|); and scores summed in fp32, whose error d (dim + 8 roundings
    of sum |q||k| * scale) changes each weight and their sum by at most
    exp(2d) - 1."""
    tokens, heads, dim = q.shape
    pages, _, kv_heads, page, _ = cache.shape
    group = heads // kv_heads
    out = np.zeros((tokens, heads, dim))
    bound = np.full((tokens, heads, dim), half_ulp16(0))
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        length = int(lens[b])
        ids = np.array([int(table[b, i]) for i in range(-(-length // page))], dtype=np.int64)
        there = np.repeat((ids >= 0) & (ids < pages), page)[:length]
        ids = np.where((ids >= 0) & (ids < pages), ids, 0)
        for h in range(kv_heads):
            if not len(ids):
                continue
            code = cache[ids][:, :, h].astype(np.float64) * scale_kv[ids][:, :, h].astype(np.float64)[..., None, None]
            k, v = code[:, 0].reshape(-1, dim)[:length], code[:, 1].reshape(-1, dim)[:length]
            for i in range(n):
                pos = length - n + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < 0:
                    continue
                see = np.arange(lo, pos + 1)
                see = see[there[lo:pos + 1]]
                if not len(see):
                    continue
                rows = q[cu[b] + i, h * group:(h + 1) * group].astype(np.float64)
                x = rows @ k[see].T * scale
                p = np.exp(x - x.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                o = p @ v[see]
                d = (np.abs(rows) @ np.abs(k[see]).T).max(axis=1, keepdims=True) * abs(scale) * (dim + 8) * 2.0 ** -24
                at = cu[b] + i, slice(h * group, (h + 1) * group)
                out[at] = o
                bound[at] = half_ulp16(np.abs(o)) * 1.001 + (p @ np.abs(v[see])) * (2.0 ** -11 + np.expm1(2 * d) + 2.0 ** -19)
    return out, bound
