"""q8_rope and q8_rope_append against the definition in 64 bits (angles modulo a turn exactly,
in whole numbers, for far positions).

Tolerances, from the arithmetic: the angle is cut to 2^-32 turns and rounded to 2^-25 half turns,
so it is off by 2^-23 radians; sine and cosine are off by 2^-23 more, their product with
the factor by 2^-24, two products and a sum by 3 * 2^-24: together below 2^-20 of
factor (|x1| + |x2|).  bf16 rounds by 2^-8 of the value.  Dimensions that pass are exact before that.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def reference(x, positions, inv_freq, interleaved, factor):
    """(y, what an error of 2^-20 is relative to), x [T, heads, D] in 64 bits."""
    from block_quantized_int8_gb300 import q8
    turns = q8.rope_turns(inv_freq, device="cpu").numpy()
    n = len(inv_freq)
    a = np.empty((x.shape[0], 1, n))
    for t, p in enumerate(positions):
        for i in range(n):
            u = (int(p) * int(turns[i])) % 2 ** 64
            a[t, 0, i] = (u if u < 2 ** 63 else u - 2 ** 64) / 2.0 ** 64 * 2 * math.pi
    i = np.arange(n)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    y, size = x.copy(), np.zeros_like(x)
    x1, x2 = x[..., lo], x[..., hi]
    y[..., lo] = factor * (x1 * np.cos(a) - x2 * np.sin(a))
    y[..., hi] = factor * (x2 * np.cos(a) + x1 * np.sin(a))
    size[..., lo] = size[..., hi] = abs(factor) * (np.abs(x1) + np.abs(x2))
    return y, size


def rows(T, h, D, seed, kind):
    x = np.random.default_rng(seed).standard_normal((T, h, D)).astype(np.float32)
    return torch.from_numpy(x).to(kind)


POS = [0, 1, 2, 17, 4095, 100003, 262143, 2 ** 24 + 1, 2 ** 31 - 1, -1, -5000, -2 ** 31]


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 32), (128, 48), (128, 128), (256, 64), (256, 240), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_layouts_parts_and_far_positions(D, rot, interleaved, kind):
    from block_quantized_int8_gb300 import q8
    f, m = q8.rope_frequencies(rot, 10000.0, "yarn", 8.0)
    h = 3
    x = rows(len(POS), h, D, rot, kind)
    y = q8.q8_rope(x.cuda(), torch.tensor(POS, dtype=torch.int32, device="cuda"), q8.rope_turns(f), interleaved, m)
    ref, size = reference(f64(x), POS, f, interleaved, m)
    assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + 2.0 ** -20 * size)
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:].to(torch.bfloat16))
    assert torch.equal(y[0].cpu(), (x[0, :, :].float() * torch.where(torch.arange(D) < rot, m, 1.0)).to(torch.bfloat16))


@pytest.mark.parametrize("T,h", [(1, 1), (1, 40), (5, 7), (300, 64), (3, 300)])
def test_tokens_and_heads(T, h):
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(64)
    x = rows(T, h, 64, T + h, torch.float32)
    pos = np.random.default_rng(T).integers(0, 200000, T).astype(np.int32)
    y = q8.q8_rope(x.cuda(), torch.from_numpy(pos).cuda(), q8.rope_turns(f))
    ref, size = reference(f64(x), pos, f, False, 1.0)
    assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + 2.0 ** -20 * size)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_of_a_wider_projection_and_in_place(interleaved):
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(128)
    turns, pos = q8.rope_turns(f), torch.arange(100, 109, dtype=torch.int32, device="cuda")
    qkv = rows(9, 8, 128, 1, torch.bfloat16).cuda()
    before = qkv.clone()
    want = q8.q8_rope(qkv[:, 2:6], pos, turns, interleaved)
    got = q8.q8_rope(qkv[:, 2:6], pos, turns, interleaved, y=qkv[:, 2:6])
    assert torch.equal(got, want) and torch.equal(qkv[:, 2:6], want)
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 6:], before[:, 6:])


def test_turning_back():
    """A turn by -p undoes one by p, to two roundings."""
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(128)
    x = rows(4, 2, 128, 2, torch.float32).cuda()
    p = torch.tensor([3, 70000, 2 ** 30, 1], dtype=torch.int32, device="cuda")
    y = q8.q8_rope(q8.q8_rope(x, p, q8.rope_turns(f)).float(), -p, q8.rope_turns(f))
    big = x.abs().amax(-1, keepdim=True).expand_as(x)
    assert torch.all((y.float() - x).abs() <= 2.0 ** -6 * big)


def test_infinities_and_nan_stay_in_their_pairs():
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(64)
    x = rows(3, 2, 64, 3, torch.float32)
    x[1, 0, 5], x[2, 1, 40] = np.inf, np.nan
    y = f64(q8.q8_rope(x.cuda(), torch.tensor([9, 9, 9], dtype=torch.int32, device="cuda"), q8.rope_turns(f)))
    bad = ~np.isfinite(y)
    want = np.zeros_like(bad)
    want[1, 0, [5, 37]] = want[2, 1, [8, 40]] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("D,rot,interleaved", [(64, 16, False), (64, 16, True), (64, 64, False), (128, 128, False), (128, 64, True),
                                               (128, 48, False), (256, 256, False), (256, 128, True)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_append_turns_and_writes(D, rot, interleaved, kind):
    from block_quantized_int8_gb300 import q8
    f, m = q8.rope_frequencies(rot, 500000.0, "yarn", 4.0)
    T, h, kv, ps, pages = 21, 6, 3, 16, 5
    r = np.random.default_rng(D + rot)
    qkv = rows(T, h + 2 * kv, D, rot, kind).cuda()
    slots = r.permutation(pages * ps)[:T].astype(np.int64)
    slots[[2, 9]] = -1
    slots[5] = pages * ps + 3
    pos = r.integers(0, 300000, T).astype(np.int32)
    planes = [torch.full((pages, kv, ps, n), 3, dtype=t, device="cuda") for n, t in ((D, torch.int8), (D // 32, torch.float16)) * 2]
    cache = q8.KvCache(*planes)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sd, pd = torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda()
    y = q8.q8_rope_append(qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:], cache, pd, sd, q8.rope_turns(f), interleaved, m, dev_status=st)
    assert int(st.item()) == q8.Q8_DEV_BAD_INDEX
    # the queries are q8_rope's, bit for bit
    assert torch.equal(y, q8.q8_rope(qkv[:, :h], pd, q8.rope_turns(f), interleaved, m))
    # the values are q8_kv_append's, bit for bit; the keys a half scale from the definition
    other = q8.KvCache.empty(pages, ps, kv, D)
    good = torch.from_numpy(np.where(slots < pages * ps, slots, -1)).cuda()
    q8.q8_kv_append(other, qkv[:, h:h + kv], qkv[:, h + kv:], good)
    kg, vg = q8.q8_kv_read(cache, good)
    _, vw = q8.q8_kv_read(other, good)
    assert torch.equal(vg, vw)
    live = (slots >= 0) & (slots < pages * ps)
    ref, size = reference(f64(qkv[:, h:h + kv]), pos, f, interleaved, m)
    top = np.repeat(np.abs(ref).reshape(T, kv, -1, 32).max(-1), 32, -1)
    big = np.repeat(size.reshape(T, kv, -1, 32).max(-1), 32, -1)
    off = np.abs(f64(kg) - ref)
    assert np.all(off[live] <= ((0.5 / 127 + 2.0 ** -11) * top + 2.0 ** -19 * big + 2.0 ** -18)[live])
    assert torch.all(kg[torch.from_numpy(~live).cuda()] == 0)
    # nothing else was written
    untouched = np.ones((pages, ps), dtype=bool)
    untouched[slots[live] // ps, slots[live] % ps] = False
    for plane in planes:
        assert torch.all(plane.transpose(1, 2)[torch.from_numpy(untouched).cuda()] == 3)


def test_append_of_keys_that_do_not_turn_is_the_plain_append():
    """At position 0 with factor 1, and past `rot`, keys are what q8_kv_append writes, bit for bit."""
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(32)
    for kind in (torch.float32, torch.bfloat16):
        qkv = rows(40, 9, 128, 5, kind).cuda()
        slots = torch.arange(40, device="cuda")
        a, b = q8.KvCache.empty(3, 16, 4, 128), q8.KvCache.empty(3, 16, 4, 128)
        for c in (a, b):
            for t in (c.kq, c.ks, c.vq, c.vs):
                t.zero_()
        q8.q8_rope_append(qkv[:, :1], qkv[:, 1:5], qkv[:, 5:], a, torch.zeros(40, dtype=torch.int32, device="cuda"), slots, q8.rope_turns(f))
        q8.q8_kv_append(b, qkv[:, 1:5], qkv[:, 5:], slots)
        for n in ("kq", "ks", "vq", "vs"):
            assert torch.equal(getattr(a, n), getattr(b, n)), (kind, n)


def test_append_flags_what_it_cannot_store():
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(64)
    x = rows(2, 3, 64, 6, torch.float32)
    x[0, 1, 3] = np.nan
    x[1, 2, 40] = 3e38
    cache = q8.KvCache.empty(1, 16, 1, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = x.cuda()
    q8.q8_rope_append(x[:, :1], x[:, 1:2], x[:, 2:], cache, torch.tensor([4, 5], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, 1], device="cuda"), q8.rope_turns(f), dev_status=st)
    assert int(st.item()) == q8.Q8_DEV_NONFINITE | q8.Q8_DEV_SCALE_OVF
    k, v = q8.q8_kv_read(cache, torch.tensor([0, 1], device="cuda"))
    assert torch.all(k[0] == 0) and torch.all(v[1, 0, 32:] == 0) and torch.any(v[1, 0, :32] != 0)


def test_no_tokens():
    from block_quantized_int8_gb300 import q8
    f, _ = q8.rope_frequencies(64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert q8.q8_rope(torch.empty((0, 2, 64), device="cuda"), none, q8.rope_turns(f)).shape == (0, 2, 64)
    e = torch.empty((0, 1, 64), device="cuda")
    y = q8.q8_rope_append(e, e, e, q8.KvCache.empty(1, 16, 1, 64), none, none.long(), q8.rope_turns(f))
    assert y.shape == (0, 1, 64)
