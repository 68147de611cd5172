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


@pytest.mark.parametrize("softcap", [2.0 ** 38, 2.0 ** 40, 1e30, 3.0e38])
def test_a_cap_far_above_the_scores_is_none(softcap):
    lens, table = [300, 17], np.arange(40).reshape(2, 20)
    cache, kv, vv = attn.filled_cache(40, 16, 1, 128, 5)
    q = attn.bf16_of(np.random.default_rng(2).standard_normal((2, 3, 128)) * 2.0).cuda()
    attn.check(cache, kv, vv, q, table, lens, softcap=softcap)


@pytest.mark.parametrize("softcap,scale", [(1e-45, 1.0), (1e-30, 1.0), (0.0, 3.0e38), (1e-40, -3.0e38)])
def test_scores_of_zero_stay_zero_however_small_the_cap(softcap, scale):
    # tokens with a key of zeros: their score is zero and counts like any other's
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = attn.filled_cache(8, 16, 1, 64, 6)
    cache.kq.zero_()
    q = attn.bf16_of(np.random.default_rng(3).standard_normal((1, 2, 64)) * 2.0 ** 100).cuda()
    attn.check(cache, 0.0 * kv, vv, q, np.arange(8).reshape(1, 8), [100], softcap=softcap, scale=scale)
