"""q8_attn_decode and q8_moe without a workspace of the caller's: they zero the words that the
kernels count with and no more, whatever the memory held before."""
import numpy as np
import pytest
import torch

import test_gpu_attn as attn
import test_gpu_moe as moe

pytestmark = pytest.mark.gpu


def call_of(which):
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(2)
    if which == "attn":
        cache, _, _ = attn.filled_cache(300, 16, 2, 128, 5)
        q = attn.bf16_of(r.standard_normal((2, 16, 128))).cuda()
        table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
        lens = torch.tensor([2400, 700], dtype=torch.int32, device="cuda")
        return (lambda ws=None: q8.q8_attn_decode(q, cache, table, lens, ws=ws), q8.q8_attn_decode_workspace_size(2, 16, 2, 128),
                q8.Q8_ATTN_ZEROED_BYTES)
    dev = [torch.from_numpy(a).cuda() for a in moe.experts(24, 512, 512, 1)]
    x, lg = torch.randn(20, 512, device="cuda").to(torch.bfloat16), torch.randn(20, 24, device="cuda")
    return lambda ws=None: q8.q8_moe(x, lg, *dev, 4, ws=ws), q8.q8_moe_workspace_size(20, 24, 512, 512, 4), q8.Q8_MOE_ZEROED_BYTES


@pytest.mark.parametrize("which", ["attn", "moe"])
def test_only_the_counters_need_zeroing(which):
    from block_quantized_int8_gb300 import q8
    call, need, zeroed = call_of(which)
    want = [t.clone() for t in call(q8.workspace(need))]
    for fill in (0xFF, 0x3C):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        ws[:zeroed] = 0
        assert all(torch.equal(a, b) for a, b in zip(call(ws), want))
        # without one: on memory that was in use for something else
        for _ in range(3):
            junk = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            del junk
            assert all(torch.equal(a, b) for a, b in zip(call(), want))


@pytest.mark.parametrize("which", ["attn", "moe"])
def test_no_more_is_zeroed(which, monkeypatch):
    from block_quantized_int8_gb300 import q8
    call, need, zeroed = call_of(which)
    monkeypatch.setattr(q8, "workspace", None)   # which would zero all of it
    assert need > 4 * zeroed
    call()
    torch.cuda.synchronize()


def test_zeroing_a_part():
    from block_quantized_int8_gb300 import q8
    ws = torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert q8.lib().q8_workspace_zero(ws.data_ptr(), 1000, side.cuda_stream) == q8.Q8_OK
    torch.cuda.synchronize()
    assert not ws[:1000].any() and bool((ws[1000:] == 7).all())
    assert q8.lib().q8_workspace_zero(None, 0, None) == q8.Q8_OK
    assert q8.lib().q8_workspace_zero(None, 16, None) == q8.Q8_ERR_ARG
