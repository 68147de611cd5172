"""The Q8_0 key-value cache (q8_kv_append, q8_kv_read: bit for bit against the
oracle's quantizer) and the attention over it (q8_attn_decode) against the
binary64 definition.

Attention tolerances, from the arithmetic: the result is rounded once to bf16
(2^-8 relative at most); every weight and every dequantised value is rounded to
binary16 (2^-11 each, so 2^-10 of sum p|v|, and 2^-25 per weight below the
normal range); scores carry fp32 sums of D / 32 blocks, below 2^-18 of
sum|q k| * scale, which moves a weight and the lse by as much.
"""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu


def bf16_of(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def filled_cache(pages, ps, heads, D, seed, spread=1.0):
    """A cache of random Q8_0 blocks; returns (cache, k values, v values) with values in binary64."""
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(seed)
    planes = []
    for _ in range(2):
        c = r.integers(-127, 128, (pages, heads, ps, D), dtype=np.int8)
        s = (r.uniform(0.2, 1.0, (pages, heads, ps, D // 32)) * spread / 64).astype(np.float16).view(np.uint16)
        planes.append((c, s))
    t = [torch.from_numpy(a).cuda() for c, s in planes for a in (c, s.view(np.int16))]
    t = [x.view(torch.float16) if x.dtype == torch.int16 else x for x in t]
    return q8.KvCache(*t), ref.values(*planes[0]), ref.values(*planes[1])


def check(cache, kv, vv, q, table, lens, scale=None, softcap=0.0, window=0, stream=None, status=0, skip_pages=()):
    from block_quantized_int8_gb300 import q8
    B, H, D = q.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = torch.from_numpy(table.astype(np.int32)).cuda()
    ln = torch.from_numpy(np.asarray(lens, dtype=np.int32)).cuda()
    torch.cuda.synchronize()
    out, lse = q8.q8_attn_decode(q, cache, tab, ln, scale=scale, softcap=softcap, window=window, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    out, lse, qn = f64(out), f64(lse), f64(q)
    sc = D ** -0.5 if scale is None else scale
    group = H // cache.kv_heads
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * cache.page_size)
        for h in range(H):
            pos = np.arange(n)
            pg = table[b][pos // cache.page_size] if n else np.zeros(0, dtype=int)
            keep = ~np.isin(pg, skip_pages) if n else np.zeros(0, dtype=bool)
            if window:
                keep &= pos >= n - window
            pg, off = pg[keep], pos[keep] % cache.page_size
            k, v = kv[pg, h // group, off], vv[pg, h // group, off]
            o, e, pv, big = ref.attention(qn[b, h], k, v, sc, softcap)
            if k.shape[0] == 0:
                assert np.all(out[b, h] == 0) and lse[b, h] == -np.inf
                continue
            fine = 2.0 ** -18 * (1 + big)
            assert abs(lse[b, h] - e) <= fine, (b, h, lse[b, h], e)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * fine) * pv + k.shape[0] * 2.0 ** -25 * np.abs(v).max(0) + 1e-30
            bad = np.abs(out[b, h] - o) > tol
            assert not bad.any(), (b, h, n, np.abs(out[b, h] - o).max(), tol.min())
    return out, lse


def run_case(D, kv_heads, group, ps, lens, window=0, softcap=0.0, seed=0, scale=None, **kw):
    B = len(lens)
    width = max(1, -(-max(lens) // ps))
    cache, kv, vv = filled_cache(B * width + 3, ps, kv_heads, D, seed)
    r = np.random.default_rng(seed + 1)
    table = r.permutation(B * width + 3)[:B * width].reshape(B, width)
    q = bf16_of(r.standard_normal((B, kv_heads * group, D)) * 1.5).cuda()
    return check(cache, kv, vv, q, table, lens, window=window, softcap=softcap, scale=scale, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 16, 20])
def test_heads_and_groups(D, group):
    run_case(D, 2, group, 16, [77, 1, 300], seed=D + group)


@pytest.mark.parametrize("ps", [16, 32, 64, 1024])
def test_page_sizes_and_tile_ends(ps):
    # lengths at, before and after tile (16), unit (64) and page ends
    run_case(128, 2, 4, ps, [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0, 1000], seed=ps)


@pytest.mark.parametrize("D,group,window,softcap", [(64, 9, 0, 0.0), (64, 16, 50, 0.0), (64, 32, 0, 20.0), (128, 12, 0, 0.0),
                                                    (128, 16, 100, 30.0), (128, 20, 0, 0.0)])
def test_groups_of_tables_for_long_sequences(D, group, window, softcap):
    # a table wide enough for 16 heads to share a pass (without a window), whatever the lengths are
    lens = [0, 77, 1, 2300, 64]
    cache, kv, vv = filled_cache(5 * 3 + 2, 1024, 2, D, D + group)
    r = np.random.default_rng(group)
    table = np.full((5, 1100 // 16 + 1), -1)
    table[:, :3] = r.permutation(17)[:15].reshape(5, 3)
    q = bf16_of(r.standard_normal((5, 2 * group, D)) * 1.5).cuda()
    check(cache, kv, vv, q, table, lens, window=window, softcap=softcap)


def test_one_token_and_none():
    run_case(128, 3, 2, 16, [0, 1, 0], seed=3)
    run_case(64, 1, 1, 16, [0], seed=4)


def test_long_sequence_is_split_and_joined():
    run_case(128, 1, 4, 64, [20011], seed=5)
    run_case(64, 2, 1, 16, [9000, 3, 5001], seed=6)


@pytest.mark.parametrize("window", [1, 16, 17, 100, 4096])
def test_window(window):
    run_case(128, 2, 3, 32, [5, 100, 257, 1025, 0], window=window, seed=window)


@pytest.mark.parametrize("softcap", [1.0, 30.0])
def test_softcap(softcap):
    run_case(256, 2, 2, 16, [300, 40], softcap=softcap, seed=7)


def test_growing_scores_move_the_reference():
    # each later tile's scores are larger: the running reference moves many times
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(40, 16, 1, 128, 8)
    s = cache.ks.float().cpu().numpy()
    s[:] = (np.arange(40 * 16).reshape(40, 1, 16, 1) * 2e-5 + 1e-4)
    s16 = s.astype(np.float16)
    cache.ks.copy_(torch.from_numpy(s16).cuda())
    cache.kq.fill_(100)
    kv = ref.values(cache.kq.cpu().numpy(), s16.view(np.uint16))
    q = bf16_of(np.full((1, 4, 128), 1.25)).cuda()
    check(cache, kv, vv, q, np.arange(40).reshape(1, 40), [640], scale=0.25)


def test_large_value_scales():
    # s * code beyond binary16's range: the tile takes scaled-down values
    cache, kv, vv = filled_cache(8, 16, 2, 128, 9)
    s = cache.vs.float().cpu().numpy()
    s[3] = 60000.0
    s[5] = 700.0
    s16 = s.astype(np.float16)
    cache.vs.copy_(torch.from_numpy(s16).cuda())
    vv = ref.values(cache.vq.cpu().numpy(), s16.view(np.uint16))
    q = bf16_of(np.random.default_rng(1).standard_normal((1, 4, 128))).cuda()
    from block_quantized_int8_gb300 import q8
    out, lse = q8.q8_attn_decode(q, cache, torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8),
                                 torch.tensor([128], dtype=torch.int32, device="cuda"))
    o, l = f64(out), f64(lse)
    k = kv.transpose(1, 0, 2, 3).reshape(2, 128, 128)
    v = vv.transpose(1, 0, 2, 3).reshape(2, 128, 128)
    for h in range(4):
        # finite, although 127 * 60000 is far above 65504; bf16 holds it
        want, e, pv, big = ref.attention(f64(q)[0, h], k[h // 2], v[h // 2], 128 ** -0.5)
        assert np.all(np.abs(o[0, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * pv + 128 * 2.0 ** -16)


def test_tiny_and_huge_queries():
    for mag in (1e-30, 1e-6, 1e4):
        cache, kv, vv = filled_cache(6, 16, 1, 128, 10, spread=0.01)
        q = bf16_of(np.random.default_rng(2).standard_normal((1, 2, 128)) * mag).cuda()
        check(cache, kv, vv, q, np.arange(6).reshape(1, 6), [90], scale=0.05)


def test_what_lies_past_a_length_does_not_matter():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(8, 32, 2, 128, 11)
    q = bf16_of(np.random.default_rng(3).standard_normal((2, 4, 128))).cuda()
    table = np.array([[0, 1, 2, 3], [4, 5, 99, -7]])   # entries past a length are not read
    lens = [100, 33]
    a = check(cache, kv, vv, q, table, lens)
    for page, off in ((3, 4), (5, 1)):
        for s in (cache.ks, cache.vs):
            s[page, :, off:] = float("nan")
        cache.vq[page, :, off:] = -128
    b = check(cache, kv, vv, q, table, lens)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_window_leaves_out_nan_before_it():
    cache, kv, vv = filled_cache(8, 16, 1, 64, 12)
    q = bf16_of(np.random.default_rng(3).standard_normal((1, 4, 64))).cuda()
    a = check(cache, kv, vv, q, np.arange(8).reshape(1, 8), [120], window=37)
    for s in (cache.ks, cache.vs):   # token 83 is the first seen: 120 - 37
        s[:5] = float("nan")
        s[5, :, :3] = float("inf")
    b = check(cache, kv, vv, q, np.arange(8).reshape(1, 8), [120], window=37)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_pages_and_lengths_outside_the_cache_are_left_out_and_flagged():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(4, 16, 1, 128, 13)
    q = bf16_of(np.random.default_rng(4).standard_normal((1, 2, 128))).cuda()
    check(cache, kv, vv, q, np.array([[0, 4, -1, 3]]), [64], status=q8.Q8_DEV_BAD_INDEX, skip_pages=(4, -1))
    check(cache, kv, vv, q, np.array([[0, 1, 2, 3]]), [65], status=q8.Q8_DEV_BAD_INDEX)
    check(cache, kv, vv, q, np.array([[0, 1, 2, 3]]), [-3], status=q8.Q8_DEV_BAD_INDEX)
    check(cache, kv, vv, q, np.array([[9, 9, 9, 9]]), [64], status=q8.Q8_DEV_BAD_INDEX, skip_pages=(9,))


def test_strided_queries_and_another_stream():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(20, 16, 2, 128, 14)
    r = np.random.default_rng(5)
    wide = bf16_of(r.standard_normal((3, 12 * 128))).cuda()   # q is a part of a wider row
    q = wide[:, 256:256 + 8 * 128].view(3, 8, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    check(cache, kv, vv, q, r.permutation(20)[:18].reshape(3, 6), [96, 50, 1], stream=s)


def test_repeats_and_graph_replays_with_other_lengths():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(300, 16, 2, 128, 15)
    q = bf16_of(np.random.default_rng(6).standard_normal((2, 8, 128))).cuda()
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150)
    lens = torch.tensor([2400, 700], dtype=torch.int32, device="cuda")
    ws = q8.workspace(q8.q8_attn_decode_workspace_size(2, 8, 2, 128))
    out, lse = q8.q8_attn_decode(q, cache, table, lens, ws=ws)
    first = out.clone()
    for _ in range(20):
        q8.q8_attn_decode(q, cache, table, lens, out=out, lse=lse, ws=ws)
        assert torch.equal(out, first)
    assert not ws[:4096].any()   # the counters are left zero
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q8.q8_attn_decode(q, cache, table, lens, out=out, lse=lse, ws=ws)
    for n in ([2400, 700], [5, 2399], [0, 0]):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        want, want_lse = q8.q8_attn_decode(q, cache, table, lens)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_many_sequences():
    r = np.random.default_rng(7)
    lens = r.integers(0, 90, 333)
    lens[[0, 5, 6, 332]] = 0
    run_case(64, 1, 2, 16, lens.tolist(), seed=16)


# ---------------------------------------------------------------------------
def kv_rows(r, T, heads, D, dtype):
    x = r.standard_normal((T, heads, D)).astype(np.float32) * r.uniform(0.01, 8, (T, heads, 1)).astype(np.float32)
    x[0, 0, :32] = 0
    x[-1, -1, :32] = np.float32(1e-41)          # below every scale: codes and scale zero
    t = torch.from_numpy(x).to(dtype)
    return t.cuda(), t.float().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,heads,D,ps", [(1, 1, 64, 16), (1, 12, 128, 16), (7, 3, 256, 64), (333, 5, 64, 32), (1025, 2, 128, 1024)])
def test_append_and_read_are_exact(oracle, dtype, T, heads, D, ps):
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(T + D)
    pages = -(-T // ps) + 2
    cache = q8.KvCache(*(torch.full(s, 77, dtype=d, device="cuda") for s, d in
                         [((pages, heads, ps, D), torch.int8), ((pages, heads, ps, D // 32), torch.float16)] * 2))
    (k, kn), (v, vn) = kv_rows(r, T, heads, D, dtype), kv_rows(r, T, heads, D, dtype)
    slots = r.permutation(pages * ps)[:T].astype(np.int64)
    if T > 5:
        slots[[1, 4]] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ts = torch.from_numpy(slots).cuda()
    q8.q8_kv_append(cache, k, v, ts, dev_status=st)
    got = q8.q8_kv_read(cache, ts, dev_status=st)
    low = q8.q8_kv_read(cache, ts, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    live = slots >= 0
    untouched = np.ones(pages * ps, dtype=bool)
    untouched[slots[live]] = False
    for x, codes, scales, y, z in ((kn, cache.kq, cache.ks, got[0], low[0]), (vn, cache.vq, cache.vs, got[1], low[1])):
        cq, sq, _ = oracle.quantize_rows(np.ascontiguousarray(x.reshape(-1, D)))
        cq, sq = cq.reshape(T, heads, D), sq.reshape(T, heads, D // 32)
        pc = codes.cpu().numpy().transpose(0, 2, 1, 3).reshape(-1, heads, D)
        ps_ = bits(scales).reshape(pages, heads, ps, D // 32).transpose(0, 2, 1, 3).reshape(-1, heads, D // 32)
        assert np.array_equal(pc[slots[live]], cq[live]) and np.array_equal(ps_[slots[live]], sq[live])
        assert np.all(pc[untouched] == 77)
        want = ref.values(cq, sq)
        want[~live] = 0
        assert np.array_equal(f64(y), want)
        assert np.array_equal(bits(z), oracle.f64_to_bf16(want).reshape(z.shape))


def test_append_flags_bad_values_and_slots(oracle):
    from block_quantized_int8_gb300 import q8
    cache = q8.KvCache.empty(2, 16, 1, 64)
    x = np.random.default_rng(1).standard_normal((4, 64)).astype(np.float32)
    x[0, 3] = np.nan
    x[1, 40] = 127.0 * 65520.0
    k = torch.from_numpy(x).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 31, 32, 5], dtype=torch.int64, device="cuda")
    q8.q8_kv_append(cache, k, k, slots, dev_status=st)
    got, _ = q8.q8_kv_read(cache, slots)
    torch.cuda.synchronize()
    assert int(st.item()) == q8.Q8_DEV_NONFINITE | q8.Q8_DEV_SCALE_OVF | q8.Q8_DEV_BAD_INDEX
    cq, sq, _ = oracle.quantize_rows(x)
    want = ref.values(cq, sq)
    want[2] = 0
    assert np.array_equal(f64(got)[:, 0], want)


def test_append_from_a_wider_row_and_empty(oracle):
    from block_quantized_int8_gb300 import q8
    cache = q8.KvCache.empty(4, 16, 2, 64)
    qkv = torch.randn(5, 3 * 128 + 64, device="cuda")
    slots = torch.tensor([9, 3, 60, 17, 18], dtype=torch.int64, device="cuda")
    q8.q8_kv_append(cache, qkv[:, 128:256], qkv[:, 256:384], slots)
    k, v = q8.q8_kv_read(cache, slots)
    for got, part in ((k, qkv[:, 128:256]), (v, qkv[:, 256:384])):
        cq, sq, _ = oracle.quantize_rows(np.ascontiguousarray(part.cpu().numpy()))
        assert np.array_equal(f64(got).reshape(5, 128), ref.values(cq, sq))
    q8.q8_kv_append(cache, qkv[:0, :128], qkv[:0, :128], slots[:0])
    assert q8.q8_kv_read(cache, slots[:0])[0].shape == (0, 2, 64)
