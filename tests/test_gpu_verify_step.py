"""The operators of a verified decoding step together: the example's model, with
prompts that share pages, drafted trees, forks and a compaction, against a plain
float64 decoder over the text that was confirmed."""
import os
import subprocess
import sys

import numpy as np
import pytest

from gpu_util import device, log
from test_gpu_decoder_layer import ROOT, plain_layer

pytestmark = pytest.mark.gpu


def plain_hidden(model, tokens, table):
    """Hidden states of a text, all layers, float64."""
    x = model.embed[tokens].double().cpu().numpy()
    for layer in model.layers:
        x = plain_layer(layer, x, table, [0, len(tokens)], [None])
    return x


def check_pages(model):
    """refs count the table's names, and the page that a row writes next is its own."""
    table, lens, refs = (t.cpu().numpy() for t in (model.table, model.lens, model.refs))
    named = np.bincount(table[table >= 0], minlength=len(refs))
    assert (named == refs).all()
    for row, n in zip(table, lens):
        assert (row[:-(-n // model.page)] >= 0).all()


def test_steps_match_a_plain_decoder():
    """What the layers add to every node's embedding, over several steps.  As with
    the plain layers each rounding to int8 is off by 0.7 % of a row's rms (half a
    step of 1/127 of its largest, uniform: 3 sigma / 127 / sqrt(12)).  A layer makes
    five, and up to three more of keys and values each time a page's scale grows or a
    confirmed token moves between pages; 2 layers and 6 steps are at most 46
    roundings, which add like independent ones to 0.7 % * sqrt(46) = 4.7 %.  A wrong
    mask, position, page or scale is off by far more."""
    import torch
    import speculative_decode as ex
    dev = device()
    log("verified steps")
    vocab, page, max_len = 512, 16, 256
    model = ex.Model(2, 512, 1024, 8, 2, 64, vocab, 120, page, max_len, dev)
    table = model.cos_sin.cpu().numpy().astype(np.float64)
    rng = np.random.default_rng(11)
    numbers = lambda n: torch.from_numpy(rng.random(n).astype(np.float32)).to(dev)
    settings = dict(temperature=0.5, top_k=20, top_p=0.95)
    prompts = [rng.integers(vocab, size=n).tolist() for n in (37, 1, 64, 150)]
    first = model.prefill(prompts, numbers(4), **settings).tolist()
    texts = [p + [t] for p, t in zip(prompts, first)]
    parents = model.parents.tolist()
    confirmed = 0

    def step():
        nonlocal confirmed
        before = model.tokens.tolist()
        drafted, hidden, path, count = model.step(numbers(len(texts) * model.nodes), **settings)
        torch.cuda.synchronize()
        drafted = drafted.cpu().numpy().reshape(len(texts), -1)
        hidden = hidden.double().cpu().numpy().reshape(len(texts), model.nodes, -1)
        worst = 0.0
        for b, text in enumerate(texts):
            assert drafted[b, 0] == text[-1] == before[b]
            for leaf in range(model.nodes - 6, model.nodes):       # the last level: every path
                nodes = [leaf]
                while parents[nodes[0]] >= 0:
                    nodes.insert(0, parents[nodes[0]])
                want = plain_hidden(model, text[:-1] + drafted[b, nodes].tolist(), table)[-len(nodes):]
                embedded = model.embed[drafted[b, nodes].tolist()].double().cpu().numpy()
                err = np.linalg.norm(hidden[b, nodes] - want, axis=1) / np.linalg.norm(want - embedded, axis=1)
                worst = max(worst, err.max())
            kept = path[b, :int(count[b])].tolist()
            assert kept[0] == 0 and all(parents[n] == m for m, n in zip(kept, kept[1:]))
            text += drafted[b, kept[1:]].tolist() + [int(model.tokens[b])]
            confirmed += len(kept) - 1
            assert int(model.lens[b]) == len(text) - 1
        log(f"largest relative error of a node {worst:.4f}")
        assert worst < 0.047
        check_pages(model)

    model.fork([0, 1, 1, 2, 3, 3])
    texts = [list(texts[i]) for i in (0, 1, 1, 2, 3, 3)]
    step()
    step()
    model.fork([5, 0, 2, 2])                                       # answers end, one continues twice
    texts = [list(texts[i]) for i in (5, 0, 2, 2)]
    check_pages(model)
    step()
    model.compact()
    check_pages(model)
    used = int((model.refs > 0).sum())
    assert bool((model.refs[:used] > 0).all())
    step()
    step()
    step()
    log(f"{confirmed} drafted tokens confirmed")
    assert confirmed > 0                                            # moves of confirmed tokens were seen


def test_captured_steps_are_the_eager_ones():
    import torch
    import speculative_decode as ex
    dev = device()
    log("captured steps")
    settings = dict(temperature=0.7, top_p=0.9)
    numbers = torch.rand(5, 3 * 16, generator=torch.Generator("cuda").manual_seed(3), device=dev)

    def start():
        model = ex.Model(1, 512, 1024, 8, 2, 64, 512, 40, 32, 160, dev)
        model.prefill([[1, 2, 3], list(range(40)), [9] * 64], numbers[0, :3].contiguous(), **settings)
        return model

    eager, replayed = start(), start()
    u = numbers[0].clone()
    assert eager.nodes == 16
    # both take the first step alike; the second is captured, which does not run it
    eager.step(u, **settings)
    replayed.step(u, **settings)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.step(u, **settings)
    for i in range(1, 5):
        u.copy_(numbers[i])
        graph.replay()
        eager.step(u, **settings)
        torch.cuda.synchronize()
        for name in ("tokens", "lens", "table", "refs"):
            assert torch.equal(getattr(eager, name), getattr(replayed, name)), (i, name)
        for a, b in zip(eager.layers, replayed.layers):
            assert torch.equal(a.cache, b.cache) and torch.equal(a.scale, b.scale)


def test_example_runs():
    device()
    log("example")
    res = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "speculative_decode.py"), "--layers", "1",
                          "--prompts", "2", "--answers", "3", "--prompt", "100", "--steps", "4", "--hidden", "1024",
                          "--inner", "2048", "--heads", "8", "--kv-heads", "2", "--vocab", "2048"],
                         capture_output=True, text=True, timeout=110)
    assert res.returncode == 0, res.stderr[-2000:]
    assert "tokens valid: True" in res.stdout
