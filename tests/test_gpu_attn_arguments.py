"""Arguments of q8_attn_decode at the ends of their ranges."""
import numpy as np
import pytest
import torch

import test_gpu_attn as attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 16, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1])
def test_a_window_that_says_unbounded(window):
    # the same answer as without one, split over as many CTAs (a split of its own would round elsewhere)
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = attn.filled_cache(700, 16, 2, 64, 3)
    q = attn.bf16_of(np.random.default_rng(1).standard_normal((2, 4, 64))).cuda()
    table = torch.arange(700, dtype=torch.int32, device="cuda").view(2, 350)
    lens = torch.tensor([5600, 3333], dtype=torch.int32, device="cuda")
    want = q8.q8_attn_decode(q, cache, table, lens)
    got = q8.q8_attn_decode(q, cache, table, lens, window=window)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    attn.check(cache, kv, vv, q, table.cpu().numpy(), [5600, 3333], window=window)
