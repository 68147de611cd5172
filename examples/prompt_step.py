"""Prompts, chunks of prompts and single tokens through a small transformer on Q8_0 weights, one
step for all of them.

A step takes a ragged batch -- any number of new tokens for each sequence, up to `rows` in all --
through its layers: pages, slots and positions on the device (q8_kv_plan), the residual's addition
and the norm (q8_rms_norm), QKV (q8_gemm), rotary positions with the write of keys and values into a
paged Q8_0 cache (q8_rope_append), attention of the new tokens over each sequence's cache
(q8_attn_chunk), the output projection and a SwiGLU MLP (q8_gemm).  Weights are random.

Lengths, pages and positions stay on the device, so the step is captured once as a CUDA graph and
replayed for a prompt, a chunk of one, or a token for each sequence.

    python examples/prompt_step.py [--prompt 300] [--steps 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_quantized_int8_gb300 import q8  # noqa: E402


class PromptStep:
    def __init__(self, batch, rows, layers=2, hidden=512, heads=8, kv_heads=2, head_dim=64, ffn=1024, vocab=4096, page=16,
                 max_len=512, seed=0):
        self.batch, self.rows, self.heads, self.kv_heads, self.head_dim, self.ffn = batch, rows, heads, kv_heads, head_dim, ffn
        self.page, self.width = page, -(-max_len // page)
        self.pages = batch * self.width
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weights(n, k):  # Q8_0 of random rows
            return q8.q8_quantize_rows(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)

        self.layers = []
        for _ in range(layers):
            self.layers.append({
                "norms": [1.0 + 0.1 * torch.randn(hidden, generator=g, device="cuda") for _ in range(2)],
                "qkv": weights((heads + 2 * kv_heads) * head_dim, hidden), "out": weights(hidden, heads * head_dim),
                "up": weights(2 * ffn, hidden), "down": weights(hidden, ffn),
                "cache": q8.KvCache.empty(self.pages, page, kv_heads, head_dim)})
        self.last_norm = torch.ones(hidden, device="cuda")
        self.embedding = torch.randn((vocab, hidden), generator=g, device="cuda")
        freq, self.factor = q8.rope_frequencies(head_dim, 10000.0, "yarn", 4.0)
        self.turns = q8.rope_turns(freq)

        def ints(n, v=0, dtype=torch.int32):
            return torch.full((n,) if isinstance(n, int) else n, v, dtype=dtype, device="cuda")
        # pages are taken from this list as sequences grow
        self.free = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)
        self.free_count, self.table = ints(1, self.pages), ints((batch, self.width), -1)
        self.lens, self.new, self.tokens = ints(batch), ints(batch), ints(rows)
        self.starts, self.slots, self.positions = ints(batch + 1), ints(rows, -1, torch.int64), ints(rows)
        self.status = ints(1)
        self.ws = q8.workspace(q8.q8_attn_chunk_workspace_size(heads, kv_heads, head_dim))
        self.attn = torch.zeros((rows, heads, head_dim), dtype=torch.bfloat16, device="cuda")
        # (rows of no sequence keep what an earlier step wrote there; their hidden states are nobody's)
        self.queries = None

    def __call__(self):
        """One step over self.new tokens of each sequence, in order in self.tokens: lengths, pages and caches
        are updated.  Returns the rows' normed hidden states, bf16 [rows, hidden]."""
        h, kv, d, st = self.heads, self.kv_heads, self.head_dim, self.status
        q8.q8_kv_plan(self.table, self.lens, self.new, self.page, self.pages, self.rows, self.free, self.free_count, self.free_count,
                      self.starts, self.slots, self.positions, self.lens, dev_status=st)
        x = self.embedding[self.tokens.to(torch.int64)]
        add = torch.zeros_like(x)
        for layer in self.layers:
            n, _, _ = q8.q8_rms_norm(add, layer["norms"][0], residual=x, dev_status=st)
            qkv = q8.q8_gemm(*layer["qkv"], n, dev_status=st).view(self.rows, h + 2 * kv, d)
            self.queries = q8.q8_rope_append(qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:], layer["cache"], self.positions, self.slots,
                                             self.turns, factor=self.factor, dev_status=st)
            q8.q8_attn_chunk(self.queries, layer["cache"], self.table, self.lens, self.starts, out=self.attn, ws=self.ws, dev_status=st)
            add = q8.q8_gemm(*layer["out"], self.attn.view(self.rows, h * d), dev_status=st)
            n, _, _ = q8.q8_rms_norm(add, layer["norms"][1], residual=x, dev_status=st)
            gate, up = q8.q8_gemm(*layer["up"], n, dev_status=st).float().split(self.ffn, 1)
            add = q8.q8_gemm(*layer["down"], (gate * torch.sigmoid(gate) * up).to(torch.bfloat16), dev_status=st)
        return q8.q8_rms_norm(add, self.last_norm, residual=x, dev_status=st)[0]

    def put(self, tokens):
        """The next step's new tokens: a list for each sequence."""
        flat = [t for s in tokens for t in s]
        assert len(tokens) == self.batch and len(flat) <= self.rows
        self.new.copy_(torch.tensor([len(s) for s in tokens], dtype=torch.int32))
        self.tokens[:len(flat)].copy_(torch.tensor(flat, dtype=torch.int32))

    def captured(self):
        """The step as a CUDA graph (after one of no tokens, which loads what it calls)."""
        self.new.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hidden = self()
        return graph, hidden


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--steps", type=int, default=32)
    a = p.parse_args()
    if not 1 <= a.prompt <= 400 or not 1 <= a.steps <= 100:
        p.error("a prompt of 1 to 400 tokens, 1 to 100 steps")
    step = PromptStep(4, 512)
    graph, hidden = step.captured()
    g = torch.Generator()
    g.manual_seed(1)
    words = torch.randint(0, 4096, (4, 512), generator=g).tolist()

    def run(tokens):
        step.put(tokens)
        graph.replay()
        torch.cuda.synchronize()
    t = time.perf_counter()
    run([words[0][:a.prompt], words[1][:7], [], words[3][:50]])
    t1 = time.perf_counter()
    for i in range(a.steps):
        run([[words[b][500 - i]] for b in range(4)])
    t2 = time.perf_counter()
    assert int(step.status.item()) == 0, "device status set"
    print("lengths", step.lens.tolist(), "pages left", int(step.free_count.item()))
    print("first step %.0f us, then %.0f us a step" % ((t1 - t) * 1e6, (t2 - t1) / a.steps * 1e6))


if __name__ == "__main__":
    main()
