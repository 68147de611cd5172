"""The stream that a call is given: as an object, as a handle, and as handle 0, the default stream."""
import numpy as np
import pytest
import torch

import test_gpu_attn as attn
import test_gpu_moe as moe

pytestmark = pytest.mark.gpu


def test_what_a_call_allocates_is_ordered_on_its_stream():
    from block_quantized_int8_gb300 import q8
    side, other = torch.cuda.Stream(), torch.cuda.Stream()

    def current():
        return torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(other):
        assert q8._new(side, current) == side.cuda_stream
        assert q8._new(side.cuda_stream, current) == side.cuda_stream
        assert q8._new(0, current) == 0
        assert q8._new(torch.cuda.default_stream(), current) == 0
        assert current() == other.cuda_stream


def test_calls_on_the_default_stream_from_within_another():
    # the workspaces are zeroed on the stream that the kernels run on
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = attn.filled_cache(150, 16, 2, 128, 4)
    q = attn.bf16_of(np.random.default_rng(1).standard_normal((1, 8, 128))).cuda()
    table = torch.arange(150, dtype=torch.int32, device="cuda").view(1, 150)
    lens = torch.tensor([2400], dtype=torch.int32, device="cuda")
    want = q8.q8_attn_decode(q, cache, table, lens)
    dev = [torch.from_numpy(a).cuda() for a in moe.experts(4, 64, 64, 1)]
    x, lg = torch.randn(3, 64, device="cuda").to(torch.bfloat16), torch.randn(3, 4, device="cuda")
    y = q8.q8_moe(x, lg, *dev, 2)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(torch.cuda.Stream()):
            a, b = q8.q8_attn_decode(q, cache, table, lens, stream=0), q8.q8_moe(x, lg, *dev, 2, stream=0)
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(a + b, want + y))
