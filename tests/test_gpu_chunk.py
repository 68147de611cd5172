"""q8_attn_chunk against the binary64 definition.

Tolerances, from the arithmetic: a key s * code is rounded to binary16 (2^-11 of it at most) and
scores are fp32 sums (below 2^-17 of sum|q k| over 256 terms), so a score is off by
fine = (2^-11 + 2^-17) max_t sum|q k_t| * scale + 2^-18; that moves the lse by as much and a
quotient of weights by twice as much.  A value s * code and a weight are rounded to binary16 (2^-11
each, and 2^-25 of the largest weight around it below the normal range); the result to bf16 (2^-8).
Over many outputs roundings do not add up like that: the 2-norm of all that a call is off
stays below 2^-8 of the result's (bf16's own rounding gives 2^-9.2 at most).
"""
import numpy as np
import pytest
import torch

from test_gpu_attn import bf16_of, f64, filled_cache

pytestmark = pytest.mark.gpu

BAD = 0x8


def definition(q, k, v, pos, keep, scale, softcap=0.0, window=0):
    """Rows q[n, D] at positions pos[n] over tokens k, v [t, D] (keep [t]: those that exist): (out, lse, sum p|v|, sum|q k|)."""
    t = np.arange(k.shape[0])
    s = q @ k.T * scale
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    seen = (t[None] <= pos[:, None]) & keep[None]
    if window:
        seen &= t[None] > pos[:, None] - window
    s = np.where(seen, s, -np.inf)
    m = s.max(-1, initial=-np.inf, keepdims=True)
    none = m[:, 0] == -np.inf
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.where(seen, np.exp(s - np.where(none[:, None], 0, m)), 0.0)
        z = e.sum(-1, keepdims=True)
        p = np.where(z > 0, e / z, 0.0)
        lse = np.where(none, -np.inf, m[:, 0] + np.log(z[:, 0]))
    big = np.where(seen, np.abs(q) @ np.abs(k).T * abs(scale), 0.0).max(-1, initial=0.0)
    top = np.where(seen.any(-1)[:, None], np.abs(v).max(0, initial=0.0)[None], 0.0)
    return p @ v, lse, p @ np.abs(v), big, top, seen.sum(-1)


def check(cache, kv, vv, q, table, lens, starts, scale=None, softcap=0.0, window=0, status=0, stream=None, want_lse=True, ws=None, tight=2.0 ** -8):
    """q bf16 [T, H, D] on the GPU; table, lens, starts as arrays.  Returns (out, lse)."""
    from block_quantized_int8_gb300 import q8
    T, H, D = q.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    tab, ln, sd = dev(table), dev(lens), dev(starts)
    mark = torch.full((T, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 5.0, device="cuda") if want_lse else None
    torch.cuda.synchronize()
    out, lse = q8.q8_attn_chunk(q, cache, tab, ln, sd, scale=scale, softcap=softcap, window=window, out=mark, lse=lse, dev_status=st,
                                stream=stream, ws=ws)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    compare(out, lse, cache, kv, vv, q, table, lens, starts, scale, softcap, window, tight)
    return out, lse


def compare(out, lse, cache, kv, vv, q, table, lens, starts, scale=None, softcap=0.0, window=0, tight=2.0 ** -8):
    T, H, D = q.shape
    ps, pages = cache.page_size, cache.pages
    table = np.asarray(table)
    sc = D ** -0.5 if scale is None else scale
    group = H // cache.kv_heads
    o, qn = f64(out), f64(q)
    l = None if lse is None else f64(lse)
    used = np.zeros(T, dtype=bool)
    off2 = ref2 = 0.0
    for b in range(len(lens)):
        s0 = min(max(int(starts[b]), 0), T)
        s1 = min(max(int(starts[b + 1]), s0), T)
        if s1 == s0:
            continue
        used[s0:s1] = True
        n = min(max(int(lens[b]), 0), table.shape[1] * ps)
        pos = n - (s1 - s0) + np.arange(s1 - s0)
        t = np.arange(n)
        pg = table[b][t // ps] if n else np.zeros(0, dtype=int)
        keep = (pg >= 0) & (pg < pages)
        pg = np.where(keep, pg, 0)
        for h in range(H):
            # what no row sees is not looked at
            lo = max(0, int(pos[0]) + 1 - window) if window else 0
            k, v = kv[pg[lo:], h // group, t[lo:] % ps], vv[pg[lo:], h // group, t[lo:] % ps]
            ref, e, pv, big, top, count = definition(qn[s0:s1, h], k, v, pos - lo, keep[lo:], sc, softcap, window)
            fine = (2.0 ** -11 + 2.0 ** -17) * big + 2.0 ** -18
            got = o[s0:s1, h]
            if l is not None:
                some = e > -np.inf
                assert np.all(l[s0:s1, h][~some] == -np.inf)
                bad = ~(np.abs(l[s0:s1, h][some] - e[some]) <= (fine + 2.0 ** -22 * np.abs(e))[some])
                assert not bad.any(), (b, h, l[s0:s1, h][some][bad][:4], e[some][bad][:4])
            tol = 2.0 ** -8 * np.abs(ref) * 1.01 + (2.0 ** -10 + 2.2 * fine)[:, None] * pv + (count * 2.0 ** -25)[:, None] * top + 1e-30
            bad = ~(np.abs(got - ref) <= tol)
            assert not bad.any(), (b, h, n, np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])
            assert np.all(got[count == 0] == 0)
            off2 += ((got - ref) ** 2).sum()
            ref2 += (ref ** 2).sum()
    assert off2 <= tight ** 2 * ref2 + 1e-60, (off2 / ref2) ** 0.5
    assert np.all(o[~used] == 5.0)
    if l is not None:
        assert np.all(l[~used] == 5.0)


def run_case(D, kv_heads, group, ps, new, lens, window=0, softcap=0.0, seed=0, pad=0, q_scale=1.5, spread=1.0, **kw):
    B = len(new)
    width = max(1, -(-max(max(lens), 1) // ps))
    r = np.random.default_rng(seed)
    cache, kv, vv = filled_cache(B * width, ps, kv_heads, D, seed, spread)
    table = r.permutation(B * width).reshape(B, width)
    starts = np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1]) + pad
    q = bf16_of(r.standard_normal((T, kv_heads * group, D)) * q_scale).cuda()
    return check(cache, kv, vv, q, table, lens, starts, window=window, softcap=softcap, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1], [200]), ([2], [2]), ([5], [300]), ([16], [16]), ([17], [33]), ([128], [128]),
                                      ([129], [129]), ([200], [777]), ([1, 2, 3, 4, 5], [1, 64, 65, 300, 5]), ([257], [300])])
def test_lengths(D, new, lens):
    run_case(D, 2, 2, 16, new, lens, seed=D + len(new) + sum(new))


@pytest.mark.parametrize("D,group", [(64, 1), (64, 3), (64, 16), (128, 1), (128, 5), (128, 7), (128, 8), (128, 32), (256, 1), (256, 3), (256, 12)])
def test_heads_that_share_keys(D, group):
    run_case(D, 2, group, 16, [37, 3, 90], [150, 3, 411], seed=group)


def test_groups_wider_than_a_row_tile():
    run_case(64, 1, 300, 16, [7, 1], [40, 90], seed=40)
    run_case(128, 2, 130, 16, [3], [300], seed=41)


def test_a_table_without_pages():
    """No page, so no length: every row sees nothing."""
    from block_quantized_int8_gb300 import q8
    cache, _, _ = filled_cache(2, 16, 1, 64, 42)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.ones((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = q8.q8_attn_chunk(q, cache, torch.empty((2, 0), dtype=torch.int32, device="cuda"), i32(3, 2), i32(0, 3, 5), return_lse=True,
                                dev_status=st)
    assert torch.all(out == 0) and torch.all(lse == -float("inf")) and int(st.item()) == BAD


def test_the_answer_may_take_the_queries_place():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(65, 64, 2, 128, 43)
    tab = torch.arange(65, dtype=torch.int32, device="cuda").view(1, 65)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = bf16_of(np.random.default_rng(43).standard_normal((90, 8, 128))).cuda()
    want, _ = q8.q8_attn_chunk(q, cache, tab, i32(4000), i32(0, 90))
    got, _ = q8.q8_attn_chunk(q, cache, tab, i32(4000), i32(0, 90), out=q)
    assert torch.equal(want, got)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256, 1024])
def test_page_sizes(ps):
    run_case(128, 3, 2, ps, [70, 1, 130], [300, 129, 1100], seed=ps)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 100, 128, 129, 1000, 2 ** 31 - 1])
def test_windows(D, window):
    run_case(D, 1, 3, 16, [150, 40, 1], [400, 40, 333], window=window, seed=window % 97)


@pytest.mark.parametrize("D,softcap,scale", [(64, 30.0, None), (128, 1.0, None), (256, 30.0, 0.2), (128, 0.0, -0.05), (128, 0.0, 0.0)])
def test_caps_and_scales(D, softcap, scale):
    run_case(D, 2, 2, 16, [50, 90], [200, 90], softcap=softcap, scale=scale, seed=3)


def test_sequences_that_take_no_part_and_rows_behind_the_last():
    run_case(128, 2, 4, 16, [0, 5, 0, 0, 33, 0], [100, 5, 0, 7, 290, 40], pad=19, seed=4)
    run_case(64, 2, 1, 16, [0, 0], [100, 5], pad=3, seed=5)


def test_many_short_sequences():
    r = np.random.default_rng(6)
    new = r.integers(0, 6, 100)
    run_case(128, 1, 4, 16, new.tolist(), (new + r.integers(0, 200, 100)).tolist(), seed=6)


@pytest.mark.parametrize("D,group,new,lens", [(128, 4, [3], [9000]), (64, 8, [20, 1], [6000, 8000]), (256, 2, [5], [5000]),
                                              (128, 1, [300], [3000]), (128, 4, [64, 64, 64], [4000, 10, 2000])])
def test_long_caches_are_split_and_joined(D, group, new, lens):
    lens = [max(a, b) for a, b in zip(new, lens)]
    run_case(D, 2, group, 64, new, lens, seed=D)


@pytest.mark.parametrize("D,group", [(64, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("batch", [512, 513, 1300])
def test_batches_past_what_is_looked_at_together(D, group, batch):
    """The list of items is made 512 sequences at a time; some of them take no part."""
    r = np.random.default_rng(batch)
    new = np.where(r.random(batch) < 0.7, r.integers(1, 4, batch), 0)
    lens = new + r.integers(0, 30, batch)
    new[700 % batch], lens[700 % batch] = 140, 500
    run_case(D, 1, group, 16, new.tolist(), lens.tolist(), seed=batch)


@pytest.mark.parametrize("seed", range(6))
def test_drawn_batches(seed):
    r = np.random.default_rng(100 + seed)
    D, kv, group, ps = int(r.choice([64, 128, 256])), int(r.integers(1, 5)), int(r.integers(1, 9)), int(r.choice([16, 64, 256]))
    batch = int(r.integers(1, 12))
    new = r.integers(0, 400 // batch + 2, batch)
    lens = new + r.integers(0, 2500, batch)
    run_case(D, kv, group, ps, new.tolist(), lens.tolist(), seed=seed, window=int(r.choice([0, 0, 333])), softcap=float(r.choice([0.0, 0.0, 20.0])),
             pad=int(r.integers(0, 9)))


def test_a_call_repeated_often_gives_the_same():
    """Two tiles of one row tile, again and again: the answer is read after the last product."""
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(26, 16, 2, 128, 31)
    tab = torch.arange(26, dtype=torch.int32, device="cuda").view(2, 13)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = bf16_of(np.random.default_rng(31).standard_normal((60, 4, 128))).cuda()
    args = (q, cache, tab, i32(200, 140), i32(0, 40, 60))
    ws = q8.workspace(q8.q8_attn_chunk_workspace_size(4, 2, 128))
    want = check(cache, kv, vv, q, tab.cpu().numpy(), [200, 140], [0, 40, 60])[0]
    for _ in range(300):
        assert torch.equal(q8.q8_attn_chunk(*args, ws=ws)[0], want)


def test_large_scores_and_a_growing_maximum():
    """Keys that grow along the sequence, so that the running maximum moves in every tile."""
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(7)
    D, n = 128, 700
    cache, kv, vv = filled_cache(44, 16, 1, D, 7)
    ramp = np.float16(0.01) * (1 + np.arange(44 * 16).reshape(44, 1, 16, 1) / 60)
    s = np.broadcast_to(ramp, (44, 1, 16, D // 32)).astype(np.float16)
    cache.ks.copy_(torch.from_numpy(np.ascontiguousarray(s)).view(cache.ks.dtype))
    kv = cache.kq.cpu().numpy().astype(np.float64) * np.repeat(s.astype(np.float64), 32, -1)
    q = bf16_of(r.standard_normal((300, 2, D)) * 2).cuda()
    check(cache, kv, vv, q, np.arange(44).reshape(1, 44), [n], [0, 300])
    assert q8


def test_equal_scores_are_a_mean():
    cache, kv, vv = filled_cache(8, 16, 1, 64, 8)
    q = torch.zeros((128, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = check(cache, kv, vv, q, np.arange(8).reshape(1, 8), [128], [0, 128])
    assert np.allclose(f64(lse)[:, 0], np.log(np.arange(1, 129)), atol=2.0 ** -20)
    assert np.allclose(f64(out)[0, 0], vv[0, 0, 0], rtol=2.0 ** -8)


def test_what_lies_past_a_length_does_not_enter():
    D, ps = 128, 16
    for lens, new in (([37, 130], [20, 7]), ([1, 16], [1, 16])):
        width = 9
        cache, kv, vv = filled_cache(2 * width, ps, 2, D, 9)
        table = np.arange(2 * width).reshape(2, width)
        q = bf16_of(np.random.default_rng(9).standard_normal((sum(new), 4, D))).cuda()
        starts = np.concatenate([[0], np.cumsum(new)])
        a, al = check(cache, kv, vv, q, table, lens, starts)
        for b, n in enumerate(lens):
            for t in range(n, width * ps):
                pg, off = table[b][t // ps], t % ps
                cache.kq[pg, :, off], cache.vq[pg, :, off] = -128, 127
                cache.ks[pg, :, off], cache.vs[pg, :, off] = float("nan"), float("inf")
        b_, bl = check(cache, kv, vv, q, table, lens, starts)
        assert torch.equal(a, b_) and torch.equal(al, bl)


def test_scales_that_are_not_finite_count_as_zero():
    D, ps = 128, 16
    cache, kv, vv = filled_cache(8, ps, 1, D, 10)
    cache.ks[2, 0, 3, 1], cache.vs[3, 0, 5, 2] = float("nan"), float("-inf")
    kv[2, 0, 3, 32:64], vv[3, 0, 5, 64:96] = 0.0, 0.0
    q = bf16_of(np.random.default_rng(10).standard_normal((90, 2, D))).cuda()
    check(cache, kv, vv, q, np.arange(8).reshape(1, 8), [128], [0, 90], status=0x1)


def test_pages_outside_the_cache_are_left_out():
    D, ps = 64, 16
    cache, kv, vv = filled_cache(20, ps, 2, D, 11)
    table = np.arange(20).reshape(2, 10)
    q = bf16_of(np.random.default_rng(11).standard_normal((60, 4, D))).cuda()
    table[0, 3], table[0, 9], table[1, 0] = -1, 20, 2 ** 31 - 1
    check(cache, kv, vv, q, table, [160, 40], [0, 40, 60], status=BAD)
    # nothing but such pages: rows that see nothing
    table[1, :] = -1
    check(cache, kv, vv, q, table, [160, 40], [0, 40, 60], status=BAD)


def test_bad_lengths_and_starts():
    D, ps = 128, 16
    cache, kv, vv = filled_cache(10, ps, 1, D, 12)
    table = np.arange(10).reshape(2, 5)
    q = bf16_of(np.random.default_rng(12).standard_normal((50, 2, D))).cuda()
    for lens, starts in (([10, 80], [0, 30, 50]), ([0, 80], [0, 30, 50]), ([-3, 80], [0, 30, 50]), ([81, 60], [0, 30, 50]),
                         ([2 ** 31 - 1, 60], [0, 30, 50]), ([60, 60], [0, 30, 51]), ([60, 60], [-4, 30, 50]), ([60, 60], [20, 10, 30]),
                         ([60, 60], [0, 2 ** 31 - 1, 50]), ([60, 60], [-2 ** 31, 10, 20])):
        check(cache, kv, vv, q, table, lens, starts, status=BAD)


def test_strided_queries_and_no_lse():
    cache, kv, vv = filled_cache(20, 16, 2, 128, 13)
    big = bf16_of(np.random.default_rng(13).standard_normal((70, 9, 128))).cuda()
    q = big[:, 3:7]
    check(cache, kv, vv, q, np.arange(20).reshape(1, 20), [300], [0, 70], want_lse=False)


def test_infinities_and_nan_stay_in_their_rows():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(20, 16, 2, 128, 14)
    q = bf16_of(np.random.default_rng(14).standard_normal((70, 4, 128))).cuda()
    tab = torch.arange(20, dtype=torch.int32, device="cuda").view(1, 20)
    ln, st = torch.tensor([300], dtype=torch.int32, device="cuda"), torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    a, _ = q8.q8_attn_chunk(q, cache, tab, ln, st)
    q[3, 1, 7], q[40, 2, 9] = float("inf"), float("nan")
    b, _ = q8.q8_attn_chunk(q, cache, tab, ln, st)
    same = (a == b).all(-1)
    assert not torch.isfinite(b[40, 2]).any()
    same[3, 1] = same[40, 2] = True
    assert bool(same.all())


@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_at_the_end_of_their_range(D, which):
    """Scales of 512 and more: s * code passes binary16's end.  Tiles that hold one keep values to 2^-16 (and weights
    to 2^-16 of the largest): what is held against them says so."""
    r = np.random.default_rng(15)
    cache, kv, vv = filled_cache(20, 16, 1, D, 15)
    for name, plane in (("k", cache.ks), ("v", cache.vs)):
        if which in (name, "both"):
            s = plane.cpu().numpy().view(np.float16).copy()
            s[7:9] = r.uniform(400, 60000, s[7:9].shape).astype(np.float16)
            plane.copy_(torch.from_numpy(s).view(plane.dtype))
    kv, vv = (q.cpu().numpy().astype(np.float64) * np.repeat(s.cpu().numpy().view(np.float16).astype(np.float64), 32, -1)
              for q, s in ((cache.kq, cache.ks), (cache.vq, cache.vs)))
    q = bf16_of(r.standard_normal((60, 2, D)) * (1e-6 if which != "v" else 1.0)).cuda()
    check(cache, kv, vv, q, np.arange(20).reshape(1, 20), [300], [0, 60])


@pytest.mark.parametrize("q_scale", [1e-30, 1e-10, 1e10, 1e30])
def test_queries_of_any_size(q_scale):
    run_case(128, 1, 2, 16, [40], [200], q_scale=q_scale, scale=0.09 / q_scale, seed=16)


def test_small_scales_are_exact():
    """Subnormal scales: products with codes are whole numbers of 2^-24, which binary16 holds."""
    run_case(128, 1, 2, 16, [40], [200], spread=1e-5, q_scale=1e4, seed=17)


def test_a_call_repeats_bit_for_bit_and_rows_do_not_depend_on_their_neighbours():
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(130, 64, 2, 128, 18)
    q = bf16_of(np.random.default_rng(18).standard_normal((200, 8, 128))).cuda()
    tab = torch.arange(130, dtype=torch.int32, device="cuda").view(1, 130)
    ln, st = torch.tensor([8000], dtype=torch.int32, device="cuda"), torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    a, al = q8.q8_attn_chunk(q, cache, tab, ln, st, return_lse=True)
    for _ in range(5):
        b, bl = q8.q8_attn_chunk(q, cache, tab, ln, st, return_lse=True)
        assert torch.equal(a, b) and torch.equal(al, bl)


def test_a_chunk_in_one_or_in_pieces():
    """Rows of one call against the same rows in two calls (the cache holds all tokens): within the tolerances of both."""
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(40, 16, 2, 128, 19)
    q = bf16_of(np.random.default_rng(19).standard_normal((300, 4, 128))).cuda()
    tab = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    whole, _ = q8.q8_attn_chunk(q, cache, tab, i32(600), i32(0, 300))
    first, _ = q8.q8_attn_chunk(q[:111], cache, tab, i32(411), i32(0, 111))
    second, _ = q8.q8_attn_chunk(q[111:], cache, tab, i32(600), i32(0, 189))
    both = torch.cat((first, second)).float()
    assert float((whole.float() - both).norm()) <= 2.0 ** -7 * float(both.norm())


def test_one_new_token_is_the_decode_call():
    from block_quantized_int8_gb300 import q8
    for D in (64, 128, 256):
        cache, kv, vv = filled_cache(40, 16, 2, D, 20)
        q = bf16_of(np.random.default_rng(20).standard_normal((4, 6, D))).cuda()
        tab = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10)
        ln = torch.tensor([1, 160, 77, 0], dtype=torch.int32, device="cuda")
        a, al = q8.q8_attn_decode(q, cache, tab, ln, window=90)
        st = torch.tensor([0, 1, 2, 3, 3], dtype=torch.int32, device="cuda")
        b, bl = q8.q8_attn_chunk(q[:3], cache, tab, ln, st, window=90, return_lse=True)
        assert float((a[:3].float() - b.float()).norm()) <= 2.0 ** -7 * float(b.float().norm())
        assert torch.allclose(al[:3], bl, atol=2e-2)


def test_graph_replay_with_other_lengths():
    from block_quantized_int8_gb300 import q8
    D, H = 128, 4
    cache, kv, vv = filled_cache(3 * 20, 16, 1, D, 21)
    r = np.random.default_rng(21)
    tables = np.arange(60).reshape(3, 20)
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    ln, st = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    q = bf16_of(r.standard_normal((200, H, D))).cuda()
    out, lse = torch.empty((200, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((200, H), device="cuda")
    ws = q8.workspace(q8.q8_attn_chunk_workspace_size(H, 1, D))
    q8.q8_attn_chunk(q, cache, tab, ln, st, out=out, lse=lse, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q8.q8_attn_chunk(q, cache, tab, ln, st, out=out, lse=lse, ws=ws)
    for lens, starts in (([300, 7, 100], [0, 100, 107, 200]), ([0, 0, 0], [0, 0, 0, 0]), ([1, 1, 1], [0, 1, 2, 3]), ([320, 320, 320], [0, 1, 1, 199]),
                         ([199, 0, 0], [0, 199, 199, 199])):
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        st.copy_(torch.tensor(starts, dtype=torch.int32))
        out.fill_(5.0)
        lse.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        compare(out, lse, cache, kv, vv, q, tables, lens, starts)


def test_streams():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run_case(128, 2, 2, 16, [50, 9], [300, 90], seed=22)
    run_case(128, 2, 2, 16, [50, 9], [300, 90], seed=22, stream=s)


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own, many times over."""
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(130, 64, 2, 128, 23)
    tab = torch.arange(130, dtype=torch.int32, device="cuda").view(1, 130)
    r = np.random.default_rng(23)
    jobs = []
    for n, t in ((64, 8000), (300, 3000)):
        q = bf16_of(r.standard_normal((t and n, 8, 128))).cuda()
        a = (q, cache, tab, torch.tensor([t], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        jobs.append((a, q8.q8_attn_chunk(*a)[0], torch.cuda.Stream(), q8.workspace(q8.q8_attn_chunk_workspace_size(8, 2, 128))))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for a, _, s, ws in jobs:
            with torch.cuda.stream(s):
                got.append(q8.q8_attn_chunk(*a, ws=ws)[0])
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, jobs[i % 2][1])


def test_one_workspace_for_all_calls():
    """The chunk's, the decode's and a matmul's workspace may be one, in stream order."""
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(130, 64, 2, 128, 24)
    r = np.random.default_rng(24)
    tab = torch.arange(130, dtype=torch.int32, device="cuda").view(1, 130)
    q = bf16_of(r.standard_normal((30, 8, 128))).cuda()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    args = (q, cache, tab, i32(8000), i32(0, 30))
    want, _ = q8.q8_attn_chunk(*args)
    dec = (q[:1], cache, tab, i32(8000))
    dwant, _ = q8.q8_attn_decode(*dec)
    w = torch.randn(4096, 1536, device="cuda")
    wq, wsc = q8.q8_quantize_rows(w)
    x = torch.randn(16, 1536, device="cuda").to(torch.bfloat16)
    ywant = q8.q8_gemm_skinny(wq, wsc, x)
    ws = torch.full((max(q8.q8_attn_chunk_workspace_size(8, 2, 128), q8.q8_attn_decode_workspace_size(1, 8, 2, 128), 1 << 24),), 0,
                    dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(q8.q8_attn_chunk(*args, ws=ws)[0], want)
        assert torch.equal(q8.q8_gemm_skinny(wq, wsc, x, ws=ws), ywant)
        assert torch.equal(q8.q8_attn_decode(*dec, ws=ws)[0], dwant)


def test_offsets_past_32_bits():
    """A cache whose codes pass 2^32 bytes: pages at both ends."""
    D, kv_heads, ps = 128, 8, 1024
    pages = 2 ** 32 // (D * kv_heads * ps) + 5
    from block_quantized_int8_gb300 import q8
    cache = q8.KvCache.empty(pages, ps, kv_heads, D)
    small, kv, vv = filled_cache(2, ps, kv_heads, D, 25)
    table = np.array([[pages - 1, 0]])
    for i, pg in enumerate(table[0]):
        for n in ("kq", "ks", "vq", "vs"):
            getattr(cache, n)[pg] = getattr(small, n)[i]

    class Far:  # kv[page, ...] for the two pages that exist
        def __init__(self, a):
            self.a = a

        def __getitem__(self, i):
            return self.a[(np.where(i[0] == 0, 1, 0),) + tuple(i[1:])]
    q = bf16_of(np.random.default_rng(25).standard_normal((20, 8, D))).cuda()
    check(cache, Far(kv), Far(vv), q, table, [1500], [0, 20])


def test_no_rows():
    from block_quantized_int8_gb300 import q8
    cache, _, _ = filled_cache(2, 16, 1, 64, 26)
    out, lse = q8.q8_attn_chunk(torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda"), cache,
                                torch.zeros((1, 2), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                                torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 64) and lse is None


@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_blocks_beside_a_scale_of_512(D):
    """A token's blocks have scales of their own.  Where one is 512 or more the token is taken times 2^-9, and what its
    other blocks hold is kept to 2^-11 of itself and 2^-16 besides: the product s * code is rounded to binary16, and
    times 2^-9 to whole multiples of 2^-24 (half of one, times 2^9).  With a window of 1 a row is its own token: out is the
    value, by one weight (2^-11) and bf16 (2^-8), and the lse is the score."""
    r = np.random.default_rng(50)
    n, ps, large = 200, 16, [3, 17, 130]
    cache, _, _ = filled_cache(13, ps, 1, D, 50)
    for plane in (cache.ks, cache.vs):
        s = (2.0 ** r.uniform(-15, -5, (13 * ps, D // 32))).astype(np.float16)
        s[17, 1:] = s[130, 1:] = 2.5 * 2.0 ** -15
        s[large, 0] = [600, 512, 40000]
        plane.copy_(torch.from_numpy(s.reshape(13, 1, ps, D // 32)).view(plane.dtype))
    k, v = (c.cpu().numpy().astype(np.float64).reshape(-1, D)[:n] * np.repeat(f64(s).reshape(-1, D // 32)[:n], 32, -1)
            for c, s in ((cache.kq, cache.ks), (cache.vq, cache.vs)))
    q = bf16_of(r.standard_normal((n, 2, D)))
    q[..., :32] = 0  # sees none of the large blocks
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    from block_quantized_int8_gb300 import q8
    out, lse = q8.q8_attn_chunk(q.cuda(), cache, torch.arange(13, dtype=torch.int32, device="cuda").view(1, 13), i32(n), i32(0, n), window=1,
                                return_lse=True)
    out, lse, qn = f64(out), f64(lse), f64(q)
    more = np.zeros((n, 1))
    more[large] = 2.0 ** -16
    for h in range(2):
        bad = ~(np.abs(out[:, h] - v) <= (2.0 ** -8 + 2.0 ** -10) * 1.01 * np.abs(v) + more)
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), out[:, h][bad][:4], v[bad][:4])
        score, big = (qn[:, h] * k).sum(-1) * D ** -0.5, (np.abs(qn[:, h]) * np.abs(k)).sum(-1) * D ** -0.5
        tol = (2.0 ** -11 + 2.0 ** -17) * big + 2.0 ** -18 + more[:, 0] * np.abs(qn[:, h]).sum(-1) * D ** -0.5
        bad = ~(np.abs(lse[:, h] - score) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), lse[:, h][bad][:4], score[bad][:4])


@pytest.mark.parametrize("D,n,lens,group", [(64, 64, 64, 1), (128, 200, 700, 1), (128, 20, 9000, 4), (256, 100, 300, 2)])
@pytest.mark.parametrize("factor", [1e9, float("nan"), float("inf"), 0.0])
def test_what_other_rows_hold_does_not_change_a_row(D, n, lens, group, factor):
    """Bit for bit, lse included, where starts and lengths are the same: every second row of the tile is made so large that
    its scores pass 2^20, or is not finite, or zero."""
    from block_quantized_int8_gb300 import q8
    pages = -(-lens // 64)
    cache, _, _ = filled_cache(pages, 64, 1, D, 51)
    q = bf16_of(np.random.default_rng(51).standard_normal((n, group, D)) * 3).cuda()
    tab = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    a, al = q8.q8_attn_chunk(q, cache, tab, i32(lens), i32(0, n), return_lse=True)
    other = q.clone()
    other[1::2] *= factor
    b, bl = q8.q8_attn_chunk(other, cache, tab, i32(lens), i32(0, n), return_lse=True)
    assert torch.equal(a[::2], b[::2]) and torch.equal(al[::2], bl[::2])


@pytest.mark.parametrize("cap", [1.0, 30.0, 255.0, 256.0, 257.0, 1000.0, 1e5, 2.0 ** 30, 2.0 ** 39, 2.0 ** 40, 3e38])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_caps_of_any_width(D, cap):
    """With a window of 1 the lse is the capped score.  Scales are powers of two and a query has one value, so that the products
    are exact and what is left is the cap's own error: 2^-21 of it where c - 2 c / (1 + 2^y) is used (exponential 2^-22,
    reciprocal 2^-23, sums 2^-24 each: 1.8 * 2^-22 of c at most), and roundings of the score (the factor's three, the product,
    and the lse: below 2^-20 of it).  The reference lies 11 below a small score: their difference, near 11, is rounded by 2^-21,
    and the weight by the exponential's 2^-22, together below 2^-20 besides.  Scores on both sides of a quarter of the cap,
    where wide caps change form."""
    r = np.random.default_rng(52)
    n, ps = 400, 16
    cache, _, _ = filled_cache(25, ps, 1, D, 52)
    cache.ks.fill_(2.0 ** -6)
    k = cache.kq.cpu().numpy().astype(np.float64).reshape(-1, D)[:n, 5] * 2.0 ** -6
    k[k == 0] = 1.0
    x = np.concatenate([r.uniform(-3, 3, 100), r.uniform(0.2, 0.3, 100) * r.choice([-1, 1], 100), 2.0 ** r.uniform(-20, 0, 200) * r.choice([-1, 1], 200)])
    want = x * min(cap, 2.0 ** 27)  # (a cap of 2^40 or more is none: it would move larger scores by more than 2^-20 of them)
    q = torch.zeros((n, 2, D), dtype=torch.bfloat16)
    q[:, :, 5] = bf16_of(want / k * D ** 0.5)[:, None]
    k = cache.kq.cpu().numpy().astype(np.float64).reshape(-1, D)[:n, 5] * 2.0 ** -6
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    from block_quantized_int8_gb300 import q8
    tab = torch.arange(25, dtype=torch.int32, device="cuda").view(1, 25)
    out, lse = q8.q8_attn_chunk(q.cuda(), cache, tab, i32(n), i32(0, n), softcap=cap, window=1, return_lse=True)
    score = f64(q)[:, :, 5] * k[:, None] * D ** -0.5
    ref = cap * np.tanh(score / cap)
    formed = (cap <= 256) | (np.abs(score / cap) > 0.249)
    tol = 2.0 ** -20 * np.abs(score) + np.where(formed, 2.0 ** -21 * cap, 0.0) + 2.0 ** -20
    bad = ~(np.abs(f64(lse) - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), f64(lse)[bad][:4], ref[bad][:4], score[bad][:4])
    v = cache.vq.cpu().numpy().astype(np.float64).reshape(-1, D)[:n] * np.repeat(f64(cache.vs).reshape(-1, D // 32)[:n], 32, -1)
    assert np.all(np.abs(f64(out) - v[:, None]) <= (2.0 ** -8 + 2.0 ** -10) * 1.01 * np.abs(v)[:, None])


@pytest.mark.parametrize("D,q_scale", [(64, 3.0), (128, 40.0), (256, 400.0)])
@pytest.mark.parametrize("softcap", [256.0, 257.0, 1000.0, 2.0 ** 40])
def test_wide_caps_of_masked_tiles(D, q_scale, softcap):
    """(Scores in the hundreds are off by more than the 2-norm's bound foresees; each output's own bound says so.)"""
    run_case(D, 2, 2, 16, [150, 3, 40], [333, 3, 401], softcap=softcap, q_scale=q_scale, seed=53, tight=1.0)
    run_case(D, 1, 3, 16, [150, 40], [400, 90], softcap=softcap, q_scale=q_scale, window=70, seed=54, tight=1.0)


@pytest.mark.parametrize("softcap", [30.0, 1000.0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_caps_and_scales_at_the_end_of_their_range(D, softcap):
    r = np.random.default_rng(55)
    cache, kv, vv = filled_cache(20, 16, 1, D, 55)
    for plane in (cache.ks, cache.vs):
        s = f64(plane).astype(np.float16)
        s[7:9] = r.uniform(400, 60000, s[7:9].shape).astype(np.float16)
        plane.copy_(torch.from_numpy(s).view(plane.dtype))
    kv, vv = (c.cpu().numpy().astype(np.float64) * np.repeat(f64(s), 32, -1) for c, s in ((cache.kq, cache.ks), (cache.vq, cache.vs)))
    q = bf16_of(r.standard_normal((60, 2, D)) * 1e-5).cuda()
    check(cache, kv, vv, q, np.arange(20).reshape(1, 20), [300], [0, 60], softcap=softcap)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("at", [5, 250])
def test_ordinary_values_beside_a_scale_of_512(D, at):
    """From a tile with a value scale of 512 or more on, a weight is good to 2^-11 of itself down to 2^-16 of the largest and to
    2^-27 of that below.  Held against the dimensions whose own scales are ordinary, with their own largest value."""
    r = np.random.default_rng(56)
    n, new = 900, 100
    cache, _, _ = filled_cache(57, 16, 1, D, 56)
    s = f64(cache.vs).astype(np.float16).reshape(57 * 16, D // 32)
    s[at, 0] = 600
    cache.vs.copy_(torch.from_numpy(s.reshape(57, 1, 16, D // 32)).view(cache.vs.dtype))
    k, v = (c.cpu().numpy().astype(np.float64).reshape(-1, D)[:n] * np.repeat(f64(s).reshape(-1, D // 32)[:n], 32, -1)
            for c, s in ((cache.kq, cache.ks), (cache.vq, cache.vs)))
    q = bf16_of(r.standard_normal((new, 2, D)) * 4)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    from block_quantized_int8_gb300 import q8
    tab = torch.arange(57, dtype=torch.int32, device="cuda").view(1, 57)
    out, _ = q8.q8_attn_chunk(q.cuda(), cache, tab, i32(n), i32(0, new))
    for h in range(2):
        ref, _, pv, big, top, count = definition(f64(q)[:, h], k, v[:, 32:], n - new + np.arange(new), np.ones(n, dtype=bool), D ** -0.5)
        fine = (2.0 ** -11 + 2.0 ** -17) * big + 2.0 ** -18
        tol = 2.0 ** -8 * 1.01 * np.abs(ref) + (2.0 ** -10 + 2.2 * fine)[:, None] * pv + (count * 2.0 ** -27)[:, None] * top + 2.0 ** -16
        bad = ~(np.abs(f64(out)[:, h, 32:] - ref) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), f64(out)[:, h, 32:][bad][:4], ref[bad][:4])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 90])
def test_the_lse_of_one_new_token_is_the_decode_calls(D, window):
    """There key codes enter exactly, here a key is rounded to binary16 (2^-11 of sum|q k|); fp32 sums are 2^-17 of it in each."""
    from block_quantized_int8_gb300 import q8
    cache, kv, vv = filled_cache(40, 16, 2, D, 57)
    q = bf16_of(np.random.default_rng(57).standard_normal((3, 6, D)) * 2)
    tables, lens = np.arange(40).reshape(4, 10)[:3], [1, 160, 77]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    tab = torch.from_numpy(tables.astype(np.int32)).cuda()
    _, al = q8.q8_attn_decode(q.cuda(), cache, tab, i32(*lens), window=window)
    _, bl = q8.q8_attn_chunk(q.cuda(), cache, tab, i32(*lens), i32(0, 1, 2, 3), window=window, return_lse=True)
    for b, n in enumerate(lens):
        t = np.arange(n)
        for h in range(6):
            k, v = (a[tables[b][t // 16], h // 3, t % 16] for a in (kv, vv))
            _, e, _, big, _, _ = definition(f64(q)[b:b + 1, h], k, v, np.array([n - 1]), np.ones(n, dtype=bool), D ** -0.5, 0.0, window)
            off = abs(float(al[b, h]) - float(bl[b, h]))
            assert off <= (2.0 ** -11 + 2.0 ** -16) * big[0] + 2.0 ** -17 + 2.0 ** -21 * abs(e[0]), (b, h, off, big)
