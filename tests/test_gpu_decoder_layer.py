"""The operators together: the example's decoder layers against a plain
float64 decoder over the same dequantized weights, prefill and decode."""
import os
import subprocess
import sys

import numpy as np
import pytest

from gpu_util import device, log

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def plain_layer(layer, x, cos_sin, starts, past):
    """One layer in float64 on x [tokens, hidden] whose rows are the sequences'
    new tokens in order; past[b] holds (k, v) of earlier tokens, extended."""
    heads, kvh, dim = layer.heads, layer.kv_heads, layer.head_dim
    rms = lambda t, w: t / np.sqrt((t * t).mean(-1, keepdims=True) + 1e-5) * w.cpu().numpy().astype(np.float64)
    mul = lambda t, lin: t @ lin.dequantized().astype(np.float64).T
    half = dim // 2
    qkv = mul(rms(x, layer.norm_in), layer.qkv).reshape(len(x), -1, dim)
    out = np.zeros((len(x), heads, dim))
    for b in range(len(past)):
        lo, hi = starts[b], starts[b + 1]
        first = 0 if past[b] is None else len(past[b][0])
        pos = np.arange(first, first + hi - lo)
        cos, sin = cos_sin[pos, None, :half], cos_sin[pos, None, half:]
        part = qkv[lo:hi].copy()
        u, v = part[:, :heads + kvh, :half].copy(), part[:, :heads + kvh, half:].copy()
        part[:, :heads + kvh, :half], part[:, :heads + kvh, half:] = u * cos - v * sin, v * cos + u * sin
        k, v = part[:, heads:heads + kvh], part[:, heads + kvh:]
        if past[b] is not None:
            k, v = np.concatenate([past[b][0], k]), np.concatenate([past[b][1], v])
        past[b] = (k, v)
        for h in range(heads):
            s = part[:, h] @ k[:, h // (heads // kvh)].T / np.sqrt(dim)
            s[np.arange(len(k))[None, :] > pos[:, None]] = -np.inf
            p = np.exp(s - s.max(axis=1, keepdims=True))
            out[lo:hi, h] = p / p.sum(axis=1, keepdims=True) @ v[:, h // (heads // kvh)]
    x = x + mul(out.reshape(len(x), -1), layer.o)
    gu = mul(rms(x, layer.norm_mlp), layer.gate_up)
    g, u = gu[:, :gu.shape[1] // 2], gu[:, gu.shape[1] // 2:]
    return x + mul(g / (1 + np.exp(-g)) * u, layer.down)


def test_layers_match_a_plain_decoder():
    """Two layers, ragged prompts, then two decode steps.  Each layer rounds
    four activations and the cache to int8; a rounding to one of 255 steps of
    a row's largest value is off by at most 1/254 of it, about 1 % of the row's
    rms for a normal row, and the errors of the ten roundings add like
    independent ones: 4 % of the output is a generous bound for their sum, and
    a wrong mask, position, page or scale is off by far more."""
    import torch
    import decoder_layer as ex
    import w4a8_gemm_amd as w4
    dev = device()
    log("decoder layers")
    hidden, inner, heads, kvh, dim = 512, 1024, 8, 2, 64
    layers = [ex.DecoderLayer(hidden, inner, heads, kvh, dim, 128, i, dev) for i in range(2)]
    prompts = [37, 1, 64, 150]
    batch = ex.Batch(prompts, 8, 16, dev)
    for layer in layers:
        layer.new_cache(batch, dev)
    cos_sin = w4.rope_table(batch.max_len, dim, device=dev)
    table = cos_sin.cpu().numpy().astype(np.float64)
    rng = np.random.default_rng(5)
    past = [[None] * len(prompts) for _ in layers]

    def check(x, starts):
        y, residual = ex.run(layers, torch.from_numpy(x).to(dev), cos_sin, batch)
        torch.cuda.synchronize()
        got = y.double().cpu().numpy() + residual.double().cpu().numpy()
        want = x.astype(np.float64)
        for layer, kv in zip(layers, past):
            want = plain_layer(layer, want, table, starts, kv)
        err = np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)
        log(f"largest relative error of a row {err.max():.4f}")
        assert err.max() < 0.04

    starts = np.concatenate([[0], np.cumsum(prompts)])
    check(rng.standard_normal((sum(prompts), hidden)).astype(np.float16), starts)
    batch.decode()
    for _ in range(2):
        batch.step()
        check(rng.standard_normal((len(prompts), hidden)).astype(np.float16), np.arange(len(prompts) + 1))


def test_example_runs():
    device()
    log("example")
    res = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"), "--layers", "1",
                          "--batch", "4", "--prompt", "100", "--steps", "4", "--hidden", "1024", "--inner", "2048",
                          "--heads", "8", "--kv-heads", "2"], capture_output=True, text=True, timeout=110)
    assert res.returncode == 0, res.stderr[-2000:]
    assert "outputs finite: True" in res.stdout
