"""Several answers to each prompt by speculative decoding, with synthetic weights:
prompts are prefilled once, answers share their pages, and in each step the model
looks at a tree of drafted tokens for every answer and keeps those that its own
samples confirm.  The step runs in a captured graph.

    python examples/speculative_decode.py [--layers 2] [--prompts 4] [--answers 4] [--steps 16]

One step:

    kv_alloc, kv_copy_pages          pages for the tree; shared ones become its own
    tree_mask                        who sees whom, and where
    layers: ... rope_append(positions) -> tree_attention ...
    rms_norm_quant -> gemm (logits) -> sample
    tree_accept, kv_keep             confirmed tokens stay in the cache

Between steps kv_fork drops answers or continues one of them several times, and
kv_compact moves the pages that are left to the front of the pool.
"""
from __future__ import annotations

import argparse
import time

import numpy as np
import torch

from decoder_layer import DecoderLayer, Linear, run
import w4a8_gemm_amd as w4


class TreeLayer(DecoderLayer):
    def attend(self, q, k, v, cos_sin, where, batch):
        if batch.mask is None:
            return super().attend(q, k, v, cos_sin, where, batch)
        q = w4.rope_append(q, k, v, cos_sin, *where, cu_q=batch.cu_q, positions=batch.positions)
        return w4.tree_attention(q, *where, batch.mask, cu_q=batch.cu_q, max_q=batch.max_q, max_len=batch.max_len)


class Step:
    """What the layers are told about a step; see decoder_layer.Batch."""

    def __init__(self, table, lens, cu_q, max_q, max_len, mask=None, positions=None):
        self.table, self.lens, self.cu_q, self.max_q, self.max_len = table, lens, cu_q, max_q, max_len
        self.mask, self.positions = mask, positions


class Model:
    """Layers, embeddings and logits.  The draft is the same model without its
    layers: its likeliest tokens depend on the last one only and stand in a table."""

    def __init__(self, layers, hidden, inner, heads, kv_heads, head_dim, vocab, pages, page, max_len, device, widths=(3, 2, 1)):
        rng = np.random.default_rng(7)
        self.layers = [TreeLayer(hidden, inner, heads, kv_heads, head_dim, 128, i, device) for i in range(layers)]
        self.embed = torch.from_numpy((4 * rng.standard_normal((vocab, hidden))).astype(np.float16)).to(device)
        self.head = Linear((rng.standard_normal((vocab, hidden)) * 2 / np.sqrt(hidden)).astype(np.float32), 128, device)
        self.norm = torch.ones(hidden, dtype=torch.float16, device=device)
        self.cos_sin = w4.rope_table(max_len, head_dim, device=device)
        self.page, self.max_len, self.device = page, max_len, device
        for layer in self.layers:
            layer.cache, layer.scale = w4.kv_cache(pages, kv_heads, head_dim, page, device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.likely = torch.cat([self.logits(rows, None).topk(max(widths), dim=1).indices
                                 for rows in self.embed.split(4096)]).int()
        # the tree: every node of a level has the next width's likeliest children
        parents, level, self.levels = [-1], [0], []
        for width in widths:
            self.levels.append((torch.tensor(level, device=device), width))
            nodes = list(range(len(parents), len(parents) + len(level) * width))
            parents += [n for n in level for _ in range(width)]
            level = nodes
        self.nodes, self.parents = len(parents), torch.tensor(parents, dtype=torch.int32, device=device)

    def logits(self, x, residual):
        _, a8, s_a = w4.rms_norm_quant(x, self.norm, residual=residual)
        return self.head.from_int8(a8, s_a)

    def copy_pages(self, src, dst, counts):
        for layer in self.layers:
            w4.kv_copy_pages(layer.cache, layer.scale, src, dst, counts)

    def prefill(self, prompts, u, **settings):
        """Prompts, lists of tokens, into the cache; their next tokens."""
        dev = self.device
        lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        table = torch.full((len(prompts), -(-self.max_len // self.page)), -1, dtype=torch.int32, device=dev)
        self.table, self.lens, self.refs, src, dst, counts = w4.kv_alloc(
            table, torch.zeros_like(lens), self.refs, lens, self.page)
        starts = np.concatenate([[0], np.cumsum([len(p) for p in prompts])])
        cu_q = torch.tensor(starts, dtype=torch.int32, device=dev)
        tokens = torch.tensor([t for p in prompts for t in p], device=dev)
        step = Step(self.table, self.lens, cu_q, max(map(len, prompts)), self.max_len)
        x, residual = run(self.layers, self.embed[tokens], self.cos_sin, step)
        last = cu_q[1:].long() - 1
        self.tokens, _ = w4.sample(self.logits(x[last], residual[last]), u, **settings)
        return self.tokens

    def fork(self, parent):
        """Row i continues answer parent[i]; nobody's pages are free again."""
        parent = torch.tensor(parent, dtype=torch.int32, device=self.device)
        self.table, self.lens, self.refs = w4.kv_fork(self.table, self.lens, self.refs, parent, self.page)
        self.tokens = self.tokens[parent.long()]

    def compact(self):
        self.table, self.refs, _, src, dst, counts = w4.kv_compact(self.table, self.refs)
        self.copy_pages(src, dst, counts)

    def draft(self):
        rows = self.tokens.shape[0]
        tokens = self.tokens.clamp(min=0).view(rows, 1)
        for level, width in self.levels:
            tokens = torch.cat([tokens, self.likely[tokens[:, level].long(), :width].reshape(rows, -1)], dim=1)
        return tokens.reshape(-1)

    def step(self, u, **settings):
        """One tree for every answer: u holds a random number for each node.
        Returns (drafted tokens, hidden states of the nodes, path, count); tokens,
        lens, table and refs are updated in place, so that a captured step can be
        replayed."""
        rows = self.tokens.shape[0]
        drafted, parents = self.draft(), self.parents.repeat(rows)
        cu_q = torch.arange(rows + 1, dtype=torch.int32, device=self.device) * self.nodes
        table, lens, refs, src, dst, counts = w4.kv_alloc(self.table, self.lens, self.refs, self.nodes, self.page)
        self.copy_pages(src, dst, counts)
        mask, positions = w4.tree_mask(parents, lens, cu_q, self.nodes)
        step = Step(table, lens, cu_q, self.nodes, self.max_len, mask, positions)
        x, residual = run(self.layers, self.embed[drafted.long()], self.cos_sin, step)
        sampled, _ = w4.sample(self.logits(x, residual), u, **settings)
        path, count, tokens, kept = w4.tree_accept(drafted, parents, sampled, lens, cu_q, self.nodes)
        for layer in self.layers:
            w4.kv_keep(layer.cache, layer.scale, table, lens, path, count, cu_q)
        for mine, new in ((self.table, table), (self.lens, kept), (self.refs, refs), (self.tokens, tokens)):
            mine.copy_(new)
        return drafted, x + residual, path, count


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("layers", 2), ("prompts", 4), ("answers", 4), ("prompt", 512), ("steps", 16), ("hidden", 4096),
                          ("inner", 14336), ("heads", 32), ("kv-heads", 8), ("head-dim", 128), ("vocab", 32000), ("page", 64)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    dev = torch.device("cuda:0")
    rng = np.random.default_rng(0)
    max_len = a.prompt + 2 * (a.steps + 4) * 4 + 16
    rows = a.prompts * a.answers
    pages = (rows + 1) * -(-max_len // a.page)
    model = Model(a.layers, a.hidden, a.inner, a.heads, a.kv_heads, a.head_dim, a.vocab, pages, a.page, max_len, dev)
    settings = dict(temperature=0.7, top_k=50, top_p=0.95)
    prompts = [rng.integers(a.vocab, size=int(n)).tolist() for n in rng.integers(max(1, a.prompt // 2), a.prompt + 1, a.prompts)]
    model.prefill(prompts, torch.rand(a.prompts, device=dev), **settings)
    model.fork([i // a.answers for i in range(rows)])

    def decode(steps):
        """Steps in a captured graph, after one that is not: (confirmed, seconds)."""
        u = torch.rand(model.tokens.shape[0] * model.nodes, device=dev)
        model.step(u, **settings)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, _, _, count = model.step(u, **settings)
        before = int(model.lens.sum())
        t = time.perf_counter()
        for _ in range(steps):
            u.uniform_()
            graph.replay()
        torch.cuda.synchronize()
        return int(model.lens.sum()) - before, time.perf_counter() - t

    def report(name, steps):
        confirmed, t = decode(steps)
        n = model.tokens.shape[0]
        print(f"{name}: {n} answers, {steps} steps of {model.nodes} nodes each: {t / steps * 1e3:.2f} ms a step, "
              f"{confirmed / steps / n:.2f} tokens confirmed in a step, {int((model.refs > 0).sum())} pages in use")

    report("decode", a.steps)
    model.fork([i * a.answers for i in range(a.prompts)])          # one answer to each prompt goes on
    model.compact()
    used = int((model.refs > 0).sum())
    assert int((model.refs[:used] > 0).sum()) == used
    report("after compaction", a.steps)
    print("tokens valid:", bool(((model.tokens >= 0) & (model.tokens < a.vocab)).all()))


if __name__ == "__main__":
    main()
