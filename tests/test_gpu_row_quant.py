"""rms_norm_quant and silu_mul_quant on the GPU against 64-bit numpy."""
import numpy as np
import pytest

import decoder_ref as dref
import w4a8_gemm_amd as w4
from gpu_util import device, log
from oracle import ref

pytestmark = pytest.mark.gpu

EPS = 1e-5
SHAPES = [(1, 1), (1, 8), (3, 7), (2, 128), (5, 130), (1, 4096), (16, 4096), (33, 5120), (257, 8192),
          (7, 14336), (64, 2056), (2, 24576), (3, 40000), (2, 40001), (1000, 264)]


def rows(m, k, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * spread
    x[:, rng.integers(0, k)] *= 20                       # an outlier channel
    return x.astype(np.float16)


def strided(a, pad, dev):
    """a on the GPU as the left part of wider rows."""
    import torch
    wide = torch.full((a.shape[0], a.shape[1] + pad), 7.0, dtype=torch.float16, device=dev)
    wide[:, :a.shape[1]] = torch.from_numpy(a).to(dev)
    return wide[:, :a.shape[1]]


def norm(x, w, res=None, **kw):
    import torch
    h, a8, s_a = w4.rms_norm_quant(x, w, EPS, residual=res, **kw)
    torch.cuda.synchronize()
    return h.cpu().numpy(), a8.cpu().numpy(), s_a.cpu().numpy()


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("m,k", SHAPES)
def test_norm(m, k, residual):
    import torch
    dev = device()
    log(f"norm m={m} k={k} residual={residual}")
    x, r = rows(m, k, 1), rows(m, k, 2, 3.0) if residual else None
    w = (1 + 0.3 * np.random.default_rng(3).standard_normal(k)).astype(np.float16)
    h, a8, s_a = norm(torch.from_numpy(x).to(dev), torch.from_numpy(w).to(dev),
                      torch.from_numpy(r).to(dev) if residual else None)
    want_h, y = dref.rms_norm(x, r, w, EPS)
    assert np.array_equal(h.view(np.uint16), want_h.view(np.uint16))
    dref.check_int8_rows(a8, s_a, y)


# every threads-and-chunks form of rows held in registers: for norm of few rows
# (one chunk a thread, then 1024 threads), of many (up to 4 chunks), the last
# chunk whole or not
FEW = [(3, 2048), (3, 4096), (2, 4104), (2, 8192), (2, 8200), (2, 16392), (1, 24584), (2, 32768)]
MANY = [(512, 2048), (513, 2056), (512, 4096), (600, 5128), (600, 8192), (512, 8200), (530, 12296),
        (512, 16384), (512, 16392), (515, 24584), (512, 32768)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("m,k", FEW + MANY)
def test_norm_held_forms(m, k, residual):
    import torch
    dev = device()
    log(f"norm held m={m} k={k} residual={residual}")
    x, r = rows(m, k, 15), rows(m, k, 16, 3.0) if residual else None
    w = (1 + 0.3 * np.random.default_rng(17).standard_normal(k)).astype(np.float16)
    h, a8, s_a = norm(torch.from_numpy(x).to(dev), torch.from_numpy(w).to(dev),
                      torch.from_numpy(r).to(dev) if residual else None)
    want_h, y = dref.rms_norm(x, r, w, EPS)
    assert np.array_equal(h.view(np.uint16), want_h.view(np.uint16))
    dref.check_int8_rows(a8, s_a, y)


@pytest.mark.parametrize("m,k", FEW + [(513, 2048), (512, 4104), (600, 8192)])
def test_silu_mul_held_forms(m, k):
    import torch
    dev = device()
    log(f"silu_mul held m={m} k={k}")
    g, u = rows(m, k, 18, 2.0), rows(m, k, 19)
    a8, s_a = w4.silu_mul_quant(torch.from_numpy(g).to(dev), torch.from_numpy(u).to(dev))
    torch.cuda.synchronize()
    dref.check_int8_rows(a8.cpu().numpy(), s_a.cpu().numpy(), dref.silu_mul(g, u), dref.FP32 + 64 * 2.0 ** -23)


@pytest.mark.parametrize("pad,into", [(8, "new"), (3, "new"), (0, "x"), (16, "residual"), (0, "residual")])
@pytest.mark.parametrize("m,k", [(6, 4096), (5, 300), (3, 33000)])
def test_norm_strides_and_in_place(m, k, pad, into):
    """Rows inside wider ones (aligned and not), and h written over x or over
    the residual."""
    import torch
    dev = device()
    log(f"norm strided m={m} k={k} pad={pad} h={into}")
    x, r = rows(m, k, 4), rows(m, k, 5, 2.0)
    w = (1 + 0.3 * np.random.default_rng(6).standard_normal(k)).astype(np.float16)
    xd, rd = strided(x, pad, dev), strided(r, pad, dev)
    out = {"new": None, "x": xd, "residual": rd}[into]
    h, a8, s_a = norm(xd, torch.from_numpy(w).to(dev), rd, h=out)
    want_h, y = dref.rms_norm(x, r, w, EPS)
    assert np.array_equal(h.view(np.uint16), want_h.view(np.uint16))
    dref.check_int8_rows(a8, s_a, y)
    if out is None:
        assert np.array_equal(xd.cpu().numpy(), x) and np.array_equal(rd.cpu().numpy(), r)
    if pad:   # what lies beside the rows stays
        whole = (out if out is not None else xd)
        beside = torch.as_strided(whole, (m, pad), (k + pad, 1), whole.storage_offset() + k)
        assert (beside == 7.0).all()


def test_norm_zero_tiny_and_large_rows():
    import torch
    dev = device()
    k = 1024
    x = rows(6, k, 7)
    x[0] = 0
    x[1] = 0
    x[1, 100] = 65504
    x[2] = (x[2].astype(np.float64) * 2.0 ** -14).astype(np.float16)     # subnormal values
    x[3] = 65504
    x[4] = -65504
    w = np.ones(k, np.float16)
    w[5] = 0
    log("norm zero, tiny and large rows")
    h, a8, s_a = norm(torch.from_numpy(x).to(dev), torch.from_numpy(w).to(dev))
    _, y = dref.rms_norm(x, None, w, EPS)
    dref.check_int8_rows(a8, s_a, y)
    assert s_a[0] == 0 and (a8[0] == 0).all()


@pytest.mark.parametrize("k", [1024, 999])
def test_norm_marks_rows_that_are_not_finite(k):
    """NaN, infinity, and a sum that overflows fp16 mark their own row only."""
    import torch
    dev = device()
    x, r = rows(6, k, 8), rows(6, k, 9)
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, 7], r[3, 7] = 60000, 60000
    log("norm non-finite rows")
    w = np.ones(k, np.float16)
    h, a8, s_a = norm(torch.from_numpy(x).to(dev), torch.from_numpy(w).to(dev),
                      torch.from_numpy(r).to(dev))
    assert np.isnan(s_a[1:4].astype(np.float32)).all()
    good = [0, 4, 5]
    want_h, y = dref.rms_norm(x[good], r[good], w, EPS)
    assert np.array_equal(h[good], want_h)
    dref.check_int8_rows(a8[good], s_a[good], y)


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("joined", [True, False])
def test_silu_mul(m, k, joined):
    import torch
    dev = device()
    log(f"silu_mul m={m} k={k} joined={joined}")
    g, u = rows(m, k, 10, 2.0), rows(m, k, 11)
    if joined:
        a8, s_a = w4.silu_mul_quant(torch.from_numpy(np.concatenate([g, u], axis=1)).to(dev))
    else:
        a8, s_a = w4.silu_mul_quant(strided(g, 24, dev), torch.from_numpy(u).to(dev))
    torch.cuda.synchronize()
    # exp's argument is rounded to fp32 before it: |g| * 2^-23 of relative error
    y = dref.silu_mul(g, u)
    dref.check_int8_rows(a8.cpu().numpy(), s_a.cpu().numpy(), y, dref.FP32 + 64 * 2.0 ** -23)


def test_silu_mul_extremes():
    import torch
    dev = device()
    k = 512
    g, u = rows(6, k, 12, 2.0), rows(6, k, 13)
    g[0, :] = -65504                                     # silu is -0
    g[1, 0] = 65504
    u[1, 0] = 1
    g[2, 9] = np.nan
    g[3, 9] = -np.inf                                    # -inf * 0
    u[4, 9] = np.inf
    g[4, 9] = 1
    g[5, :] = 0
    log("silu_mul extremes")
    a8, s_a = w4.silu_mul_quant(torch.from_numpy(g).to(dev), torch.from_numpy(u).to(dev))
    torch.cuda.synchronize()
    a8, s_a = a8.cpu().numpy(), s_a.cpu().numpy()
    assert s_a[0] == 0 and (a8[0] == 0).all() and s_a[5] == 0 and (a8[5] == 0).all()
    assert np.isnan(s_a[2]) and np.isnan(s_a[3]) and np.isinf(s_a[4])
    dref.check_int8_rows(a8[1:2], s_a[1:2], dref.silu_mul(g[1:2], u[1:2]), dref.FP32 + 64 * 2.0 ** -23)


def test_outputs_feed_the_gemm():
    """rms_norm_quant -> gemm -> silu_mul_quant -> gemm equals the same
    products of the codes, exactly."""
    import torch
    import synth
    dev = device()
    m, k, n, g = 9, 512, 1024, 128
    w_up, w_down = synth.weights(n, k, seed=3), synth.weights(k, n // 2, seed=4)
    x = rows(m, k, 14)
    log("norm -> gemm -> silu_mul -> gemm")
    xd = torch.from_numpy(x).to(dev)
    _, a8, s_a = w4.rms_norm_quant(xd, torch.ones(k, dtype=torch.float16, device=dev), EPS)
    y = w4.gemm(a8, s_a, w4.to_device(w4.pack(w_up, g), dev), n, k, g)
    b8, s_b = w4.silu_mul_quant(y)
    z, acc = w4.gemm(b8, s_b, w4.to_device(w4.pack(w_down, g), dev), k, n // 2, g, want_acc=True)
    torch.cuda.synchronize()
    qw = ref.quantize_weights(w_down, g)
    assert np.array_equal(acc.cpu().numpy(), ref.gemm_acc(b8.cpu().numpy(), ref.decoded_weights(qw)))


def test_empty_batch_and_refusals():
    import torch
    dev = device()
    x = torch.zeros((0, 64), dtype=torch.float16, device=dev)
    w = torch.ones(64, dtype=torch.float16, device=dev)
    h, a8, s_a = w4.rms_norm_quant(x, w, residual=x)
    assert h.shape == (0, 64) and a8.shape == (0, 64) and s_a.shape == (0,)
    a8, s_a = w4.silu_mul_quant(x)
    assert a8.shape == (0, 32)
    x = torch.zeros((4, 64), dtype=torch.float16, device=dev)
    with pytest.raises(ValueError):
        w4.rms_norm_quant(x.float(), w)
    with pytest.raises(ValueError):
        w4.rms_norm_quant(x, w[:32])
    with pytest.raises(ValueError):
        w4.rms_norm_quant(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        w4.rms_norm_quant(x.t(), w[:4])
    with pytest.raises(ValueError):
        w4.silu_mul_quant(x[:, :63])
    with pytest.raises(ValueError):
        w4.silu_mul_quant(x, x[:, :32])
    with pytest.raises(w4.W4A8Error) as err:
        w4.rms_norm_quant(x, w, eps=-1.0)
    assert err.value.status == 1
