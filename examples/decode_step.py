"""A decode step of a small transformer on Q8_0 weights, start to end on the library.

Every step takes the batch's last tokens through its layers -- QKV (q8_gemm_skinny), the new
keys and values into a paged Q8_0 cache (q8_kv_append), attention over each sequence's cache
(q8_attn_decode), the output projection, a router and a mixture of Q8_0 experts (q8_moe) --
then the vocabulary projection and the draw of the next tokens (q8_sample).  Norms and
residuals are plain torch.  Weights are random; there is no position encoding.

The step allocates nothing in the library and reads lengths, page numbers and knobs from the
device, so it is captured once as a CUDA graph and replayed.

    python examples/decode_step.py [--steps 32] [--batch 4]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_quantized_int8_gb300 import q8  # noqa: E402


class DecodeStep:
    def __init__(self, batch, layers=2, hidden=512, heads=8, kv_heads=2, head_dim=64, experts=8, top_k=2, ffn=256, vocab=8192,
                 page=16, max_len=256, seed=0):
        self.batch, self.hidden, self.heads, self.kv_heads, self.head_dim = batch, hidden, heads, kv_heads, head_dim
        self.experts, self.top_k, self.page, self.max_len = experts, top_k, page, max_len
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weights(*shape):  # Q8_0 of random rows
            w = torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5
            q, s = q8.q8_quantize_rows(w.view(-1, shape[-1]))
            return q.view(shape), s.view(*shape[:-1], shape[-1] // 32)

        def linear(n, k):
            q, s = weights(n, k)
            return q, s, torch.empty((batch, n), dtype=torch.float32, device="cuda"), q8.workspace(q8.q8_workspace_size(n, k, batch))

        rows = (heads + 2 * kv_heads) * head_dim
        width = -(-max_len // page)
        self.layers = []
        for _ in range(layers):
            self.layers.append({
                "qkv": linear(rows, hidden), "out": linear(hidden, heads * head_dim), "router": linear(experts, hidden),
                "q13": weights(experts, 2 * ffn, hidden), "q2": weights(experts, hidden, ffn),
                "cache": q8.KvCache.empty(batch * width, page, kv_heads, head_dim)})
        self.head = linear(vocab, hidden)
        self.embedding = torch.randn((vocab, hidden), generator=g, device="cuda")
        # a sequence's pages lie anywhere in the cache
        self.table = torch.randperm(batch * width, generator=g, device="cuda").to(torch.int32).view(batch, width)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.u = torch.zeros(batch, dtype=torch.float32, device="cuda")
        self.temperature = torch.full((batch,), 0.8, device="cuda")
        self.knob_k = torch.full((batch,), 50, dtype=torch.int32, device="cuda")
        self.knob_p = torch.full((batch,), 0.95, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.attn_ws = q8.workspace(q8.q8_attn_decode_workspace_size(batch, heads, kv_heads, head_dim))
        self.moe_ws = q8.workspace(q8.q8_moe_workspace_size(batch, experts, hidden, ffn, top_k))

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def linear(self, x, w):
        q, s, y, ws = w
        return q8.q8_gemm_skinny(q, s, x, y=y, ws=ws, dev_status=self.status)

    def __call__(self):
        """One step: reads self.tokens and self.u, appends to the cache, leaves the next tokens in
        self.tokens.  Returns their log-probabilities."""
        b, h, kv, d = self.batch, self.heads, self.kv_heads, self.head_dim
        at = self.lens.to(torch.int64)
        page = self.table.gather(1, (at // self.page).view(b, 1)).view(b).to(torch.int64)
        slots = page * self.page + at % self.page
        self.lens += 1
        x = self.embedding[self.tokens.to(torch.int64)]
        for layer in self.layers:
            qkv = self.linear(self.norm(x), layer["qkv"])
            q = qkv[:, :h * d].to(torch.bfloat16).view(b, h, d)
            q8.q8_kv_append(layer["cache"], qkv[:, h * d:(h + kv) * d], qkv[:, (h + kv) * d:], slots, dev_status=self.status)
            a, _ = q8.q8_attn_decode(q, layer["cache"], self.table, self.lens, ws=self.attn_ws, dev_status=self.status)
            x = x + self.linear(a.view(b, h * d), layer["out"])
            n = self.norm(x)
            y, _, _ = q8.q8_moe(n, self.linear(n, layer["router"]), *layer["q13"], *layer["q2"], self.top_k, ws=self.moe_ws,
                                dev_status=self.status)
            x = x + y
        logits = self.linear(self.norm(x), self.head)
        token, logprob, _ = q8.q8_sample(logits, self.u, temperature=self.temperature, top_k=self.knob_k, top_p=self.knob_p,
                                         dev_status=self.status)
        self.tokens.copy_(token)
        return logprob

    def captured(self):
        """The step as a CUDA graph (after one eager step, whose effect on the lengths is undone)."""
        before = self.lens.clone(), self.tokens.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self()
            self.lens.copy_(before[0])
            self.tokens.copy_(before[1])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logprob = self()
        return graph, logprob


def generate(step, steps, seed=1, graph=None):
    """`steps` tokens per sequence from given random numbers: (tokens [steps, batch], log-probabilities)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    tokens, logprobs = [], []
    for _ in range(steps):
        step.u.copy_(torch.rand(step.batch, generator=g, device="cuda"))
        if graph is None:
            logprobs.append(step().clone())
        else:
            graph[0].replay()
            logprobs.append(graph[1].clone())
        tokens.append(step.tokens.clone())
    return torch.stack(tokens), torch.stack(logprobs)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--batch", type=int, default=4)
    a = p.parse_args()
    if not 1 <= a.batch <= q8.Q8_SKINNY_MAX_M or not 1 <= a.steps <= 250:
        p.error("1 to 32 sequences, 1 to 250 steps")
    step = DecodeStep(a.batch)
    graph = step.captured()
    generate(step, 2, graph=graph)  # loads what the steps call
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens, logprobs = generate(step, a.steps, graph=graph)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    assert int(step.status.item()) == 0, "device status set"
    print("tokens of the first sequence:", tokens[:, 0].tolist())
    print("mean log-probability %.3f; %.1f us a step of %d sequences" % (logprobs.mean().item(), t / a.steps * 1e6, a.batch))


if __name__ == "__main__":
    main()
