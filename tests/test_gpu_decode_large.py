"""The decode-step calls where offsets pass 32 bits and at their largest widths, with the
tolerances of the tests of each call."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import test_gpu_attn as attn
import test_gpu_moe as moe
import test_gpu_sample as sample

pytestmark = pytest.mark.gpu


class Pages:
    """values[page, head, offset] of the few pages that hold any."""

    def __init__(self, pages, values):
        self.at = {p: i for i, p in enumerate(pages)}
        self.values = values

    def __getitem__(self, key):
        page, head, offset = key
        return self.values[[self.at[p] for p in page], head, offset]


def test_a_cache_of_more_than_2_32_codes(oracle):
    from block_quantized_int8_gb300 import q8
    heads, ps, D = 2, 1024, 128
    pages = 2 ** 32 // (heads * ps * D) + 16
    cache = q8.KvCache.empty(pages, ps, heads, D)
    used = [pages - 1, 0, pages // 2 + 9, pages - 7]  # around 0, 2^31 and 2^32
    T = len(used) * ps
    r = np.random.default_rng(3)
    slots = torch.from_numpy(np.concatenate([p * ps + np.arange(ps) for p in used])).cuda()
    x = [r.standard_normal((T, heads * D)).astype(np.float32) for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q8.q8_kv_append(cache, *(torch.from_numpy(a).cuda() for a in x), slots, dev_status=st)
    got = q8.q8_kv_read(cache, slots, dev_status=st)
    planes = []
    for a, g in zip(x, got):
        cq, sq, _ = oracle.quantize_rows(a)
        v = ref.values(cq, sq)
        assert np.array_equal(attn.f64(g).reshape(T, heads * D), v)
        planes.append(Pages(used, v.reshape(len(used), ps, heads, D).transpose(0, 2, 1, 3)))
    assert int(st.item()) == 0
    q = attn.bf16_of(r.standard_normal((2, heads * 3, D)) * 1.5).cuda()
    attn.check(cache, *planes, q, np.array([used, used[::-1]]), [T, T - 1500])


def test_experts_of_more_than_2_32_codes():
    from block_quantized_int8_gb300 import q8
    E, H, F, T, k = 512, 2048, 2080, 5, 2
    some = [511, 3, 260]
    c13, s13, c2, s2 = moe.experts(len(some), H, F, 8)
    dev = []
    for codes, scales in ((c13, s13), (c2, s2)):
        q = torch.empty((E, *codes.shape[1:]), dtype=torch.int8, device="cuda")
        s = torch.empty((E, *scales.shape[1:]), dtype=torch.float16, device="cuda")
        for i, e in enumerate(some):
            q[e] = torch.from_numpy(codes[i]).cuda()
            s[e] = torch.from_numpy(scales[i]).cuda()
        dev += [q, s]
    assert dev[0].numel() > 2 ** 32
    r = np.random.default_rng(9)
    x = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    few = r.standard_normal((T, len(some))).astype(np.float32)
    logits = np.full((T, E), -np.inf, dtype=np.float32)
    logits[:, some] = few
    y, ids, w = q8.q8_moe(x, torch.from_numpy(logits).cuda(), *dev, k)
    want, tol, wi, ww = ref.moe(x.double().cpu().numpy(), few, ref.values(c13, s13.view(np.uint16)), ref.values(c2, s2.view(np.uint16)),
                                k, True)
    assert np.array_equal(ids.cpu().numpy(), np.array(some)[wi])
    assert np.all(np.abs(w.double().cpu().numpy() - ww) <= 2.0 ** -20 * ww)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("T,E,H,F,k", [(3, 1, 8192, 96, 1), (9, 2, 96, 20000, 1), (32, 2, 8192, 64, 2), (32, 2, 512, 2080, 2),
                                       (3, 4, 160, 1568, 2), (1, 1, 32, 65536, 1)])
def test_the_largest_widths_of_experts(T, E, H, F, k):
    moe.run(T, E, H, F, k, seed=H + F + T)


def test_rows_of_logits_further_apart_than_2_31():
    r = np.random.default_rng(4)
    n, V, ld = 2, 5000, 2 ** 31 + 40
    logits = torch.empty(ld + V, dtype=torch.float32, device="cuda").as_strided((n, V), (ld, 1))
    logits.copy_(torch.from_numpy((r.standard_normal((n, V)) * 2.5).astype(np.float32)))
    sample.check(logits, r.random(n).astype(np.float32), k=[0, 40], p=[0.9, 1.0])


def test_queries_near_the_end_of_the_range():
    cache, kv, vv = attn.filled_cache(6, 16, 1, 128, 10)
    r = np.random.default_rng(2)
    q = attn.bf16_of(r.standard_normal((1, 2, 128)) * 2.0 ** 124).cuda()
    attn.check(cache, kv, vv, q, np.arange(6).reshape(1, 6), [90], scale=2.0 ** -126)


def test_hidden_units_near_the_end_of_the_range():
    moe.run(4, 4, 128, 128, 2, seed=5, xs=2.0 ** 61)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,heads,D", [(8193, 5, 64), (8195, 4, 128), (4099, 3, 256)])
def test_reading_many_tokens(oracle, dtype, T, heads, D):
    from block_quantized_int8_gb300 import q8
    cache = q8.KvCache.empty(-(-T // 64) + 1, 64, heads, D)
    r = np.random.default_rng(T)
    x = [torch.from_numpy(r.standard_normal((T, heads * D)).astype(np.float32)).to(dtype) for _ in range(2)]
    slots = r.permutation(T + 64)[:T].astype(np.int64)
    slots[::97] = -1
    at = torch.from_numpy(slots).cuda()
    q8.q8_kv_append(cache, *(a.cuda() for a in x), at)
    for a, g in zip(x, q8.q8_kv_read(cache, at, dtype=dtype)):
        cq, sq, _ = oracle.quantize_rows(a.float().numpy())
        want = torch.from_numpy(ref.values(cq, sq).astype(np.float32)).to(dtype)
        want[::97] = 0
        assert torch.equal(g.cpu().view(T, heads * D), want)
