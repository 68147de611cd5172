"""The decode step of examples/decode_step.py: the new operators together with the matmuls,
against the same step written plainly in binary64, and as a CUDA graph."""
import os
import sys

import numpy as np
import pytest
import torch

import decode_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def host(w):
    return ref.values(w[0].cpu().numpy(), w[1].cpu().view(torch.int16).numpy().view(np.uint16))


def norm(x):
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).double().numpy()


def bf16(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).double().numpy()


def plain_logits(step, tokens):
    """The last logits of a sequence's tokens, every step from the start, in binary64 (rounded to
    bf16 and Q8_0 where the step is)."""
    import oracle
    oracle.build()
    d, h, kv = step.head_dim, step.heads, step.kv_heads
    emb = step.embedding.double().cpu().numpy()
    past = [([], []) for _ in step.layers]
    for tok in tokens:
        x = emb[tok]
        for layer, (ks, vs) in zip(step.layers, past):
            qkv = host(layer["qkv"]) @ norm(x)
            q = bf16(qkv[:h * d]).reshape(h, d)
            for part, out in ((qkv[h * d:(h + kv) * d], ks), (qkv[(h + kv) * d:], vs)):
                c, s, _ = oracle.quantize_rows(np.ascontiguousarray(part.reshape(kv, d), dtype=np.float32))
                out.append(ref.values(c, s))
            k, v = np.stack(ks), np.stack(vs)
            a = np.stack([ref.attention(q[i], k[:, i // (h // kv)], v[:, i // (h // kv)], d ** -0.5)[0] for i in range(h)])
            x = x + host(layer["out"]) @ bf16(a.reshape(-1))
            n = norm(x)
            lg = host(layer["router"]) @ n
            y, *_ = ref.moe(n[None], lg[None].astype(np.float32), host(layer["q13"]), host(layer["q2"]), step.top_k, True)
            x = x + y[0]
    return host(step.head) @ norm(x)


def test_step_against_the_plain_one():
    import decode_step
    step = decode_step.DecodeStep(2, layers=2, hidden=128, heads=4, kv_heads=2, head_dim=64, experts=4, top_k=2, ffn=64, vocab=512,
                                  max_len=64)
    step.temperature.zero_()   # the likeliest word each time
    fed = [[0], [0]]
    for _ in range(20):
        step()
        for b in range(2):
            fed[b].append(int(step.tokens[b].item()))
    assert int(step.status.item()) == 0 and step.lens.tolist() == [20, 20]
    for b in range(2):
        got = step.head[2][b].double().cpu().numpy()
        want = plain_logits(step, fed[b][:-1])
        # a bf16 or Q8_0 rounding that falls the other way moves what follows by 2^-8 of it
        assert np.linalg.norm(got - want) <= 2.0 ** -6 * np.linalg.norm(want)
        assert fed[b][-1] == int(np.argmax(got))


def test_graph_replays_are_the_eager_steps():
    import decode_step
    eager, graphed = decode_step.DecodeStep(5), decode_step.DecodeStep(5)
    graph = graphed.captured()
    a = decode_step.generate(eager, 40)
    b = decode_step.generate(graphed, 40, graph=graph)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert int(eager.status.item()) == 0 and int(graphed.status.item()) == 0
