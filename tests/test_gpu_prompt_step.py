"""The prompt-step operators together, as examples/prompt_step.py runs them.

However a sequence's tokens are cut into steps, each row's arithmetic up to the attention is the
same (the rows of a matmul, a norm and a rotation do not see each other); the attention joins its
tiles in another order, so that a row of it may differ by a bf16 step (2^-8), and by a code of 127
of the next layer's cache through that, in each of two layers: 2 (2^-8 + 2^-7) of the hidden state, below 2^-5.
"""
import os
import sys

import numpy as np
import pytest
import torch

import test_gpu_chunk as chunk
from test_gpu_attn import f64

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def words(n, seed=3):
    return np.random.default_rng(seed).integers(0, 4096, n).tolist()


def rows_of(step, hidden):
    s = step.starts.tolist()
    return [hidden[s[b]:s[b + 1]].float().clone() for b in range(step.batch)]


def run(step, parts, graph=None):
    """Each step's list of tokens per sequence; returns each sequence's hidden states, all steps together."""
    out = [[] for _ in range(step.batch)]
    for tokens in parts:
        step.put(tokens)
        if graph is None:
            hidden = step()
        else:
            graph[0].replay()
            hidden = graph[1]
        for b, r in enumerate(rows_of(step, hidden)):
            out[b].append(r)
    assert int(step.status.item()) == 0
    return [torch.cat(o) for o in out]


def test_however_the_tokens_are_cut_into_steps():
    from prompt_step import PromptStep
    a, b, c = words(150, 1), words(90, 2), words(41, 3)
    whole = run(PromptStep(3, 300), [[a, b, c]])
    cut = run(PromptStep(3, 300), [[a[:100], b[:7], []], [a[100:149], b[7:60], c[:40]], [[], b[60:90], c[40:]], [a[149:], [], []]])
    graph_step = PromptStep(3, 300)
    graph = graph_step.captured()
    replayed = run(graph_step, [[a[:100], b[:7], []], [a[100:149], b[7:60], c[:40]], [[], b[60:90], c[40:]], [a[149:], [], []]], graph)
    for w, x, y in zip(whole, cut, replayed):
        assert torch.equal(x, y)
        assert float((w - x).norm()) <= 2.0 ** -5 * float(w.norm())


def test_a_steps_attention_and_cache_against_64_bits():
    from prompt_step import PromptStep
    from block_quantized_int8_gb300 import q8
    step = PromptStep(2, 128, layers=1)
    run(step, [[words(70, 5), words(20, 6)]])
    before = step.lens.tolist()
    step.attn.fill_(5.0)
    run(step, [[words(30, 7), words(51, 8)]])
    assert before == [70, 20] and step.lens.tolist() == [100, 71]
    # every token has a slot of its own, in a page of its own sequence
    table = step.table.cpu().numpy()
    used = table[table >= 0]
    assert len(set(used.tolist())) == len(used) == 7 + 5 and int(step.free_count.item()) == step.pages - 12
    cache = step.layers[0]["cache"]
    slots = torch.arange(step.pages * step.page, device="cuda")
    k, v = (f64(t).reshape(step.pages, step.page, step.kv_heads, step.head_dim).transpose(0, 2, 1, 3) for t in q8.q8_kv_read(cache, slots))
    chunk.compare(step.attn, None, cache, k, v, step.queries, table, step.lens.tolist(), step.starts.tolist())


def test_the_norms_8_bit_rows_are_what_w8a8_makes_of_a_row():
    """Q8_0 rows of the norm and the rows that the W8A8 product quantizes for itself stand for the same values to bf16's rounding."""
    from block_quantized_int8_gb300 import q8
    x = torch.randn(40, 512, device="cuda")
    y, q, s = q8.q8_rms_norm(x, quantized=True)
    w = torch.randn(256, 512, device="cuda") * 0.05
    wq, ws = q8.q8_quantize_rows(w)
    got = q8.q8_gemm_w8a8(wq, ws, y)
    value = lambda a, b: a.float() * b.float().repeat_interleave(32, 1)  # noqa: E731
    want = value(q, s).double() @ value(wq, ws).double().T
    # a code of x may differ by one: half a bf16 step (2^-8) of it against its block's scale
    size = value(q, s).abs().reshape(40, 16, 32).amax(-1).repeat_interleave(32, 1).double() @ value(wq, ws).abs().double().T
    assert torch.all((got.double() - want).abs() <= (1 / 127 + 2.0 ** -8) * size)
