"""Where the roundings of q8_attn_decode could show: large value scales beside small ones, and
weights far below the largest.

Bound, from the arithmetic: before it is rounded the result is within e of the binary64 one, where
a dequantised value is rounded once to binary16 (2^-11 of it), a weight too (2^-11 of it, or 2^-36 of
the largest weight where that is more), and a score's fp32 sums move a weight by less than
2^-18 (1 + sum|q k| scale) of itself, its share by twice that.  Rounding is monotone, so the bf16
result lies between the roundings of both ends."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import test_gpu_attn as attn

pytestmark = pytest.mark.gpu


def planes_to_cache(kq, ks, vq, vs):
    from block_quantized_int8_gb300 import q8
    ks, vs = ks.astype(np.float16), vs.astype(np.float16)
    cache = q8.KvCache(*(torch.from_numpy(a).cuda() for a in (kq, ks, vq, vs)))
    return cache, ref.values(kq, ks.view(np.uint16)), ref.values(vq, vs.view(np.uint16))


def check(cache, kv, vv, q, table, n):
    """One sequence of n tokens in the pages `table`, scale 1; every head against binary64."""
    from block_quantized_int8_gb300 import q8
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = q8.q8_attn_decode(q, cache, torch.tensor([table], dtype=torch.int32, device="cuda"),
                                 torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0, dev_status=st)
    out, lse, qn = attn.f64(out)[0], attn.f64(lse)[0], attn.f64(q)[0]
    assert int(st.item()) == 0
    pos = np.arange(n)
    pg, off = np.asarray(table)[pos // cache.page_size], pos % cache.page_size
    group = qn.shape[0] // cache.kv_heads
    for h in range(qn.shape[0]):
        k, v = kv[pg, h // group, off], vv[pg, h // group, off]
        o, e, pv, big = ref.attention(qn[h], k, v, 1.0)
        fine = 2.0 ** -18 * (1 + big)
        assert abs(lse[h] - e) <= fine
        s = k @ qn[h]
        d = (2.0 ** -10 + 2 * fine) * pv + 2.0 ** -36 * np.abs(v).sum(0) / np.exp(s - s.max()).sum()
        lo, hi = (torch.from_numpy(x).to(torch.bfloat16).double().numpy() for x in (o - d, o + d))
        bad = (out[h] < lo) | (out[h] > hi)
        assert not bad.any(), (h, o[bad][:4], out[h][bad][:4], lo[bad][:4], hi[bad][:4])


def tokens(D, heads, pages, ps, scores, r):
    """Keys whose score with a query of ones / 1024 is about scores[token], values of codes 64 .. 127."""
    kq = np.full((pages, heads, ps, D), 127, dtype=np.int8)
    ks = np.broadcast_to((scores * 1024.0 / (127.0 * D)).reshape(pages, 1, ps, 1), (pages, heads, ps, D // 32)).copy()
    vq = r.integers(64, 128, (pages, heads, ps, D), dtype=np.int8)
    q = torch.full((1, heads, D), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    return kq, ks, vq, q


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("large", [512.0, 600.0, 60000.0])
def test_small_value_scales_beside_large_ones(D, large):
    # one token of every tile has large values and next to no weight (2^-40): the others' digits stay
    r = np.random.default_rng(D)
    scores = np.full(16 * 16, 28.0)
    scores[3::16] = 0.25
    kq, ks, vq, q = tokens(D, 2, 16, 16, scores, r)
    vs = r.uniform(0.9, 1.1, (16, 2, 16, D // 32)) * 1.4e-4
    vs[:, :, 3] = large
    check(*planes_to_cache(kq, ks, vq, vs), q.repeat(1, 2, 1), list(range(16)), 250)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_lowest_code_at_a_scale_of_512(D):
    # 512 * -128 is beyond binary16; a cache may come from elsewhere than q8_kv_append
    r = np.random.default_rng(D)
    kq, ks, vq, q = tokens(D, 1, 4, 16, r.uniform(1.0, 2.0, 64), r)
    vq[:] = -128
    check(*planes_to_cache(kq, ks, vq, np.full((4, 1, 16, D // 32), 512.0)), q, [2, 0, 3, 1], 64)


@pytest.mark.parametrize("D,heads", [(64, 1), (128, 1), (256, 1), (64, 16), (128, 16)])
@pytest.mark.parametrize("log2", [14, 20, 23.4, 26])
def test_weights_far_below_the_largest(D, heads, log2):
    # one token of every tile has the largest weight and no value: what comes out is the others', each
    # at 2^-log2 of it (16 heads a pass where the table is long)
    r = np.random.default_rng(D)
    n = 500
    scores = np.zeros(32 * 16)
    scores[5::16] = log2 * np.log(2.0)
    kq, ks, vq, q = tokens(D, 1, 32, 16, scores + 1.0, r)
    vq[:, :, 5] = 0
    vs = np.full((32, 1, 16, D // 32), 0.01)
    table = list(range(32)) + ([-1] * (10016 * 64 // 16) if heads > 8 else [])
    check(*planes_to_cache(kq, ks, vq, vs), q.repeat(1, heads, 1), table, n)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("log2", [20, 23, 24, 24.7, 25, 25.6, 26, 26.4, 26.9, 27, 27.3, 27.8, 28, 28.5, 29, 31, 60])
def test_scores_whose_neighbours_are_further_apart_than_the_weights_range(D, log2):
    # equal scores of 2^log2 (and, in some tiles, others that are lower by 2^(log2 - 10) and do not count):
    # the mean of the values that do
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(D)
    n, pages = 700, 48
    kq = np.full((pages, 1, 16, D), 64, dtype=np.int8)
    ks = np.full((pages, 1, 16, D // 32), 0.5)
    low = np.zeros(pages * 16, dtype=bool)
    low[100:260] = True
    low[400::3] = True
    ks[low.reshape(pages, 1, 16)] *= 1 - 2.0 ** -10
    vq = r.integers(-127, 128, (pages, 1, 16, D), dtype=np.int8)
    cache, kv, vv = planes_to_cache(kq, ks, vq, np.full((pages, 1, 16, D // 32), 0.01))
    q = torch.ones((1, 4, D), dtype=torch.bfloat16, device="cuda")
    scale = float(np.float32(2.0 ** log2 * np.log(2.0) / (32.0 * D)))
    out, lse = q8.q8_attn_decode(q, cache, torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages),
                                 torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale)
    v = vv[:, 0].reshape(-1, D)[:n][~low[:n]]
    mean, size = v.mean(0), np.abs(v).mean(0)
    lo, hi = (torch.from_numpy(x).to(torch.bfloat16).double().numpy() for x in (mean - 2.0 ** -10 * size, mean + 2.0 ** -10 * size))
    got = attn.f64(out)[0]
    assert np.all((got >= lo) & (got <= hi)), (got[0][:4], mean[:4])
    want = scale * 32.0 * D + np.log(v.shape[0])
    assert np.all(np.abs(attn.f64(lse) - want) <= 2.0 ** -21 * want)


@pytest.mark.parametrize("base", [0.0, 1e-3, 40.0, 3e4, 2.0 ** 22])
def test_references_that_move_by_less_than_their_own_rounding(base):
    # scores base + 0 .. 20 in any order, large ones late in some warps and early in others
    r = np.random.default_rng(1)
    D, pages = 64, 40
    kq = np.zeros((pages, 1, 16, D), dtype=np.int8)
    kq[..., 0] = 1
    kq[..., 32] = r.integers(0, 21, (pages, 1, 16))
    ks = np.ones((pages, 1, 16, 2))
    vq = r.integers(64, 128, (pages, 1, 16, D), dtype=np.int8)
    cache, kv, vv = planes_to_cache(kq, ks, vq, np.full((pages, 1, 16, 2), 0.01))
    q = torch.zeros((1, 2, D), device="cuda")
    q[..., 0], q[..., 32] = base, 1.0
    q = q.to(torch.bfloat16)
    check(cache, kv, vv, q, r.permutation(pages).tolist(), 633)
