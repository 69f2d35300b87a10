"""Decoder layers built from the package's operators, with synthetic weights:
prompts of different lengths are prefilled into a paged int8 KV cache, then
every sequence decodes a few tokens in a captured graph.

    python examples/decoder_layer.py [--layers 2] [--batch 16] [--prompt 512] [--steps 32]

One layer:

    rms_norm_quant -> gemm (QKV) -> rope_append -> paged_attention -> linear (O)
    -> rms_norm_quant -> gemm (gate, up) -> silu_mul_quant -> gemm (down)
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a8_gemm_amd as w4  # noqa: E402


class Linear:
    """A W4A8 linear layer: y = x W^T, W packed once."""

    def __init__(self, weight: np.ndarray, g: int, device):
        self.n, self.k, self.g = *weight.shape, g
        self.packed = w4.pack(weight, g)
        self.blob = w4.to_device(self.packed, device)

    def from_int8(self, a8, s_a):
        return w4.gemm(a8, s_a, self.blob, self.n, self.k, self.g)

    def __call__(self, x):
        return w4.linear(x, self.blob, self.n, self.k, self.g)[0]

    def dequantized(self):
        """The float32 weight the codes stand for."""
        u = w4.unpack(self.packed)
        step = self.k // u["s2"].shape[1]
        wide = lambda a: np.repeat(a.astype(np.float32), step, axis=1)
        return (u["q"].astype(np.float32) - wide(u["z"])) * wide(u["s2"]) * u["s1"].astype(np.float32)[:, None]


class Batch:
    """Where each sequence's pages are and how many tokens it holds; shared by
    all layers.  Pages are handed out in order here."""

    def __init__(self, prompts, room, page, device):
        most = -(-(max(prompts) + room) // page)
        self.page, self.pages = page, most * len(prompts)
        self.table = torch.arange(self.pages, dtype=torch.int32, device=device).view(len(prompts), most)
        self.max_len = max(prompts) + room
        self.lens = torch.tensor(prompts, dtype=torch.int32, device=device)
        self.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device=device)
        self.max_q = max(prompts)

    def decode(self):
        """From here on every sequence brings one token."""
        self.cu_q, self.max_q = None, 1

    def step(self):
        self.lens.add_(1)


class DecoderLayer:
    def __init__(self, hidden, inner, heads, kv_heads, head_dim, g, seed, device):
        rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        make = lambda n, k: Linear((rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32), g, device)
        self.qkv = make((heads + 2 * kv_heads) * head_dim, hidden)
        self.o = make(hidden, heads * head_dim)
        self.gate_up = make(2 * inner, hidden)
        self.down = make(hidden, inner)
        norm = lambda: torch.from_numpy((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float16)).to(device)
        self.norm_in, self.norm_mlp = norm(), norm()

    def new_cache(self, batch: Batch, device):
        self.cache, self.scale = w4.kv_cache(batch.pages, self.kv_heads, self.head_dim, batch.page, device)

    def attend(self, q, k, v, cos_sin, where, batch: Batch):
        q = w4.rope_append(q, k, v, cos_sin, *where, cu_q=batch.cu_q)
        return w4.paged_attention(q, *where, cu_q=batch.cu_q, max_q=batch.max_q, max_len=batch.max_len)

    def __call__(self, x, residual, cos_sin, batch: Batch):
        """x is what the layer before adds to the residual stream (or the
        embeddings, residual None); returns the same pair for the next."""
        where = (self.cache, self.scale, batch.table, batch.lens)
        h, a8, s_a = w4.rms_norm_quant(x, self.norm_in, residual=residual)
        qkv = self.qkv.from_int8(a8, s_a).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        y = self.o(self.attend(q, k, v, cos_sin, where, batch).view(x.shape[0], -1))
        h, a8, s_a = w4.rms_norm_quant(y, self.norm_mlp, residual=h)
        a8, s_a = w4.silu_mul_quant(self.gate_up.from_int8(a8, s_a))
        return self.down.from_int8(a8, s_a), h


def run(layers, x, cos_sin, batch):
    residual = None
    for layer in layers:
        x, residual = layer(x, residual, cos_sin, batch)
    return x, residual


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("layers", 2), ("batch", 16), ("prompt", 512), ("steps", 32), ("hidden", 4096),
                          ("inner", 14336), ("heads", 32), ("kv-heads", 8), ("head-dim", 128), ("page", 64)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(0)
    layers = [DecoderLayer(a.hidden, a.inner, a.heads, a.kv_heads, a.head_dim, 128, i, dev)
              for i in range(a.layers)]
    prompts = [int(n) for n in rng.integers(max(1, a.prompt // 2), a.prompt + 1, a.batch)]
    batch = Batch(prompts, a.steps + 8, a.page, dev)
    for layer in layers:
        layer.new_cache(batch, dev)
    cos_sin = w4.rope_table(batch.max_len, a.head_dim, device=dev)
    x = torch.randn(sum(prompts), a.hidden, device=dev).half()

    run(layers, x, cos_sin, batch)                       # warm up; the second pass writes the same pages
    torch.cuda.synchronize()
    t = time.perf_counter()
    run(layers, x, cos_sin, batch)
    torch.cuda.synchronize()
    print(f"prefill: {sum(prompts)} tokens in {a.batch} prompts, {a.layers} layers: "
          f"{(time.perf_counter() - t) * 1e3:.2f} ms")

    batch.decode()
    token = torch.randn(a.batch, a.hidden, device=dev).half()

    def step():
        batch.step()
        return run(layers, token, cos_sin, batch)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = step()
    graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    print(f"decode: {a.batch} sequences, {a.steps} steps: "
          f"{(time.perf_counter() - t) / a.steps / a.layers * 1e6:.1f} us per step and layer, "
          f"outputs finite: {bool(torch.isfinite(y).all())}")


if __name__ == "__main__":
    main()
