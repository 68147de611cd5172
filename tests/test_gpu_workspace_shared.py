"""One workspace, or parts of it, through calls of every kind that takes one, in any order: each
result is, bit for bit, what the call gives with a workspace of its own."""
import numpy as np
import pytest
import torch

import decode_ref as ref  # noqa: F401
import test_gpu_attn as attn
import test_gpu_moe as moe

pytestmark = pytest.mark.gpu


def rows(r, *shape):
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).cuda()


def calls():
    """[(bytes, call(ws) -> tensors)]"""
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(7)
    out = []

    def weights(n, k):
        return q8.q8_quantize_rows(rows(r, n, k))

    def matmul(m, n, k, variant=q8.Q8_VARIANT_AUTO):
        q, s = weights(n, k)
        x, y = rows(r, m, k).to(torch.bfloat16), torch.empty((m, n), dtype=torch.float32, device="cuda")
        d, _ = q8.make_descs([(q, s, x, y)])
        need = int(q8.lib().q8_linear_batch_workspace_size_ex(d, 1, m, variant))

        def call(ws):
            y.fill_(float("nan"))
            q8.q8_linear_batch([(q, s, x, y)], ws=ws, variant=variant)
            return (y,)
        out.append((need, call))

    for m, n, k in ((1, 1000, 1536), (1, 300, 4096), (2, 200, 160), (4, 500, 4096), (5, 260, 2048), (12, 700, 1536), (16, 300, 2080),
                    (32, 200, 1536)):
        matmul(m, n, k)
    matmul(5, 300, 1536, q8.Q8_VARIANT_W8A8)
    matmul(9, 300, 2080, q8.Q8_VARIANT_W8A8)
    matmul(7, 300, 2080, q8.Q8_VARIANT_BATCH_INVARIANT)

    # a chain of three steps of different shapes
    steps, k = [], 512
    x = rows(r, 12, 512).to(torch.bfloat16)
    for i, n in enumerate((1536, 768, 640)):
        q, s = weights(n, k)
        steps.append((q, s, x, torch.empty((12, n), dtype=torch.float32, device="cuda"), q8.Q8_CHAIN_RMSNORM if i < 2 else q8.Q8_CHAIN_END))
        k = n
        x = torch.empty((12, n), dtype=torch.bfloat16, device="cuda")
    chain, M = q8.make_chain(steps)

    def run_chain(ws):
        steps[-1][3].fill_(float("nan"))
        q8.q8_linear_chain(chain, M, ws=ws)
        return (steps[-1][3],)
    out.append((q8.q8_linear_chain_workspace_size(chain, M), run_chain))

    # attention split over CTAs and joined, and over a group of more than 8 heads
    for D, group in ((128, 4), (64, 12)):
        cache, _, _ = attn.filled_cache(300, 16, 2, D, D)
        query = rows(r, 2, 2 * group, D).to(torch.bfloat16)
        table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
        lens = torch.tensor([2400, 700], dtype=torch.int32, device="cuda")
        o, e = torch.empty((2, 2 * group, D), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 2 * group), dtype=torch.float32, device="cuda")

        def run_attn(ws, query=query, cache=cache, table=table, lens=lens, o=o, e=e):
            o.fill_(float("nan"))
            q8.q8_attn_decode(query, cache, table, lens, out=o, lse=e, ws=ws)
            return o, e
        out.append((q8.q8_attn_decode_workspace_size(2, 2 * group, 2, D), run_attn))

    for T, E, H, F, k in ((1, 4, 256, 512, 2), (20, 24, 512, 512, 4)):
        dev = [torch.from_numpy(a).cuda() for a in moe.experts(E, H, F, T)]
        tokens, logits = rows(r, T, H).to(torch.bfloat16), rows(r, T, E)
        y = torch.empty((T, H), dtype=torch.float32, device="cuda")

        def run_moe(ws, dev=dev, tokens=tokens, logits=logits, y=y, k=k):
            y.fill_(float("nan"))
            return q8.q8_moe(tokens, logits, *dev, k, y=y, ws=ws)
        out.append((q8.q8_moe_workspace_size(T, E, H, F, k), run_moe))
    return out


@pytest.mark.parametrize("parts", [False, True])
def test_one_workspace_for_all_calls(parts):
    from block_quantized_int8_gb300 import q8
    todo = calls()
    want = []
    for need, call in todo:
        want.append([t.clone() for t in call(q8.workspace(need))])
        assert not any(t.isnan().any() for t in want[-1])
    ws = q8.workspace(max(need for need, _ in todo) + 64 * 256)
    r = np.random.default_rng(3)
    for i in np.concatenate([r.permutation(len(todo)) for _ in range(12)]):
        need, call = todo[i]
        at = 256 * int(r.integers(0, 64)) if parts else 0
        got = call(ws[at:at + need] if need else None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), (i, at)
