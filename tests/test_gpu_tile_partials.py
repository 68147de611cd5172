"""Row blocks that CTAs share out between them where one CTA takes a row block's first classes
and another the rest (the tile kernel at M = 2 .. 32): their sum takes in the partials of this
call alone, whatever earlier calls of other shapes left in the workspace."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# N and K such that a running sum goes through the second class of some row block (the first four), and others
SHAPES = [(700, 1536), (11000, 4096), (13000, 2048), (20000, 1536), (1536, 4096), (6000, 2048), (4608, 1536)]


@pytest.mark.parametrize("M", [5, 12, 16, 32])
def test_stale_partials_do_not_count(M):
    from block_quantized_int8_gb300 import q8
    g = torch.Generator(device="cuda").manual_seed(M)
    mats, fresh, need = [], [], 0
    for n, k in SHAPES:
        q, s = q8.q8_quantize_rows(torch.randn(n, k, generator=g, device="cuda"))
        x = torch.randn(M, k, generator=g, device="cuda").to(torch.bfloat16)
        mats.append((q, s, x))
        need = max(need, q8.q8_workspace_size(n, k, M))
        fresh.append(q8.q8_gemm_skinny(q, s, x))
    ws = q8.workspace(need)
    r = np.random.default_rng(M)
    for i in np.concatenate([r.permutation(len(mats)) for _ in range(8)]):
        got = q8.q8_gemm_skinny(*mats[i], ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, fresh[i]), SHAPES[i]


def test_a_row_block_shared_two_ways_against_the_definition():
    # twelve rows of 700 x 1536 after a call whose partials lie all over the workspace
    from block_quantized_int8_gb300 import q8
    g = torch.Generator(device="cuda").manual_seed(1)
    big = q8.q8_quantize_rows(torch.randn(20000, 1536, generator=g, device="cuda"))
    q, s = q8.q8_quantize_rows(torch.randn(700, 1536, generator=g, device="cuda"))
    x = torch.randn(12, 1536, generator=g, device="cuda").to(torch.bfloat16)
    ws = q8.workspace(q8.q8_workspace_size(20000, 1536, 12))
    q8.q8_gemm_skinny(*big, x * 1000.0, ws=ws)
    y = q8.q8_gemm_skinny(q, s, x, ws=ws).double()
    w = q.double() * s.double().repeat_interleave(32, 1)
    want, bound = x.double() @ w.T, x.double().abs() @ w.abs().T
    assert bool(((y - want).abs() <= 2e-3 * bound + 1e-6).all())
