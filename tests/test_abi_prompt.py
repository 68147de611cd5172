"""The prompt-step entry points refuse bad arguments on the host, before any CUDA call
(so these run without a GPU); the rotary table, which is made on the host, against exact
arithmetic."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest

from test_abi_decode import A, BAD_CACHES, cache


@pytest.fixture(scope="module")
def L():
    from block_quantized_int8_gb300 import build, q8
    build.build()
    return q8.lib()


def err(name):
    from block_quantized_int8_gb300 import q8
    return getattr(q8, "Q8_" + ("OK" if name == "OK" else "ERR_" + name))


def norm(L, x=A, ldx=64, xt=0, r=A, ldr=64, rt=0, ro=A, ldo=64, w=A, off=0.0, eps=1e-6, T=3, W=64, y=A, ldy=64, q=A, s=A, status=None):
    return L.q8_rms_norm(x, ldx, xt, r, ldr, rt, ro, ldo, w, off, eps, T, W, y, ldy, q, s, status, None)


def test_norm_validation(L):
    for kw, e in [(dict(xt=2), "ARG"), (dict(rt=-1), "ARG"), (dict(T=-1), "SHAPE"), (dict(T=1 << 31), "SHAPE"), (dict(W=0), "SHAPE"),
                  (dict(W=40), "SHAPE"), (dict(W=32800, ldx=32800, ldr=32800, ldo=32800, ldy=32800), "SHAPE"), (dict(eps=-1e-9), "ARG"),
                  (dict(eps=math.nan), "ARG"), (dict(eps=math.inf), "ARG"), (dict(off=math.inf), "ARG"), (dict(q=None), "ARG"),
                  (dict(s=None), "ARG"), (dict(r=None), "ARG"), (dict(ldx=60), "SHAPE"), (dict(ldr=60), "SHAPE"), (dict(ldo=60), "SHAPE"),
                  (dict(ldy=56), "SHAPE"), (dict(x=None), "ARG"), (dict(y=None, q=None, s=None, ro=None), "ARG"), (dict(ldx=66), "ALIGN"),
                  (dict(ldx=68, xt=1), "ALIGN"), (dict(ldr=66), "ALIGN"), (dict(ldo=65), "ALIGN"), (dict(ldy=68), "ALIGN"),
                  (dict(T=0), "OK"), (dict(T=0, x=None, y=None, q=None, s=None, ro=None), "OK")]:
        assert norm(L, **kw) == err(e), kw
    for a in ("x", "r", "ro", "w", "y", "q", "s"):
        assert norm(L, **{a: A + 8}) == err("ALIGN"), a
    assert norm(L, status=A + 2) == err("ALIGN")


def rope(L, x=A, ldx=256, t=0, y=A, ldy=256, h=2, d=128, rot=128, layout=0, f=1.0, turns=A, pos=A, T=3):
    return L.q8_rope(x, ldx, t, y, ldy, h, d, rot, layout, f, turns, pos, T, None)


def rope_append(L, c=None, q=A, ldq=512, h=4, k=A, v=A, ldk=256, ldv=256, t=0, rot=128, layout=0, f=1.0, turns=A, pos=A, slots=A, T=3,
                y=A, ldy=512, status=None):
    c = cache() if c is None else c
    return L.q8_rope_append(ctypes.byref(c) if c else None, q, ldq, h, k, v, ldk, ldv, t, rot, layout, f, turns, pos, slots, T, y, ldy,
                            status, None)


@pytest.mark.parametrize("fn", [rope, rope_append])
def test_rope_validation(L, fn):
    for kw, e in [(dict(t=2), "ARG"), (dict(layout=2), "ARG"), (dict(f=math.nan), "ARG"), (dict(f=math.inf), "ARG"), (dict(T=-1), "SHAPE"),
                  (dict(h=0), "SHAPE"), (dict(rot=0), "SHAPE"), (dict(rot=24), "SHAPE"), (dict(rot=144), "SHAPE"), (dict(turns=None), "ARG"),
                  (dict(pos=None), "ARG"), (dict(turns=A + 4), "ALIGN"), (dict(pos=A + 2), "ALIGN"), (dict(y=None), "ARG"),
                  (dict(y=A + 8), "ALIGN"), (dict(ldy=100), "SHAPE"), (dict(ldy=516), "ALIGN"), (dict(T=0), "OK")]:
        assert fn(L, **kw) == err(e), kw
    if fn is rope:
        for kw, e in [(dict(d=96), "SHAPE"), (dict(ldx=255), "SHAPE"), (dict(ldx=258), "ALIGN"), (dict(ldx=260, t=1), "ALIGN"),
                      (dict(x=None), "ARG"), (dict(x=A + 8), "ALIGN"), (dict(h=65537, ldx=1 << 30, ldy=1 << 30), "SHAPE")]:
            assert fn(L, **kw) == err(e), kw
        return
    for kw, e in BAD_CACHES:
        assert fn(L, c=cache(**kw)) == err(e), kw
    assert fn(L, c=False) == err("ARG")
    for kw, e in [(dict(ldq=511), "SHAPE"), (dict(ldq=514), "ALIGN"), (dict(ldk=255), "SHAPE"), (dict(ldv=258), "ALIGN"),
                  (dict(q=None), "ARG"), (dict(k=None), "ARG"), (dict(v=None), "ARG"), (dict(slots=None), "ARG"), (dict(slots=A + 4), "ALIGN"),
                  (dict(q=A + 8), "ALIGN"), (dict(k=A + 8), "ALIGN"), (dict(status=A + 2), "ALIGN")]:
        assert fn(L, **kw) == err(e), kw


def plan(L, table=A, width=8, pages=4, ps=16, lens=A, new=A, B=3, free=A, cap=4, count=A, left=A, T=9, starts=A, slots=A, pos=A, out=A,
         status=None):
    return L.q8_kv_plan(table, width, pages, ps, lens, new, B, free, cap, count, left, T, starts, slots, pos, out, status, None)


def test_plan_validation(L):
    for kw, e in [(dict(ps=8), "SHAPE"), (dict(ps=48), "SHAPE"), (dict(ps=2048), "SHAPE"), (dict(pages=0), "SHAPE"), (dict(width=-1), "SHAPE"),
                  (dict(width=1 << 27), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(B=(1 << 20) + 1), "SHAPE"), (dict(T=-1), "SHAPE"),
                  (dict(T=1 << 31), "SHAPE"), (dict(cap=-1), "SHAPE"), (dict(starts=None), "ARG"), (dict(lens=None), "ARG"), (dict(new=None), "ARG"),
                  (dict(out=None), "ARG"), (dict(table=None), "ARG"), (dict(slots=None), "ARG"), (dict(pos=None), "ARG"),
                  (dict(count=None), "ARG"), (dict(left=None), "ARG"), (dict(slots=A + 4), "ALIGN")]:
        assert plan(L, **kw) == err(e), kw
    for a in ("table", "lens", "new", "free", "count", "left", "starts", "pos", "out", "status"):
        assert plan(L, **{a: A + 2}) == err("ALIGN"), a


def chunk(L, c=None, q=A, ldq=1024, heads=8, T=9, table=A, width=4, lens=A, starts=A, batch=3, scale=0.1, cap=0.0, window=0, out=A, lse=A,
          ws=A, wsb=1 << 40, status=None):
    c = cache() if c is None else c
    return L.q8_attn_chunk(ctypes.byref(c) if c else None, q, ldq, heads, T, table, width, lens, starts, batch, scale, cap, window, out, lse,
                           ws, wsb, status, None)


def test_chunk_validation(L):
    for kw, e in BAD_CACHES:
        assert chunk(L, c=cache(**kw)) == err(e), kw
    assert chunk(L, c=False) == err("ARG")
    for kw, e in [(dict(heads=7), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(batch=-1), "SHAPE"), (dict(T=-1), "SHAPE"),
                  (dict(T=1 << 30), "SHAPE"), (dict(width=-1), "SHAPE"), (dict(width=1 << 27), "SHAPE"), (dict(window=-1), "ARG"),
                  (dict(cap=-1.0), "ARG"), (dict(cap=math.nan), "ARG"), (dict(cap=math.inf), "ARG"), (dict(scale=math.nan), "ARG"),
                  (dict(scale=math.inf), "ARG"), (dict(ldq=1016), "SHAPE"), (dict(ldq=1028), "ALIGN"), (dict(q=None), "ARG"),
                  (dict(table=None), "ARG"), (dict(lens=None), "ARG"), (dict(starts=None), "ARG"), (dict(out=None), "ARG"),
                  (dict(q=A + 8), "ALIGN"), (dict(out=A + 8), "ALIGN"), (dict(starts=A + 2), "ALIGN"), (dict(lens=A + 2), "ALIGN"),
                  (dict(table=A + 2), "ALIGN"), (dict(lse=A + 2), "ALIGN"), (dict(status=A + 2), "ALIGN"), (dict(ws=None), "WORKSPACE"),
                  (dict(wsb=100), "WORKSPACE"), (dict(ws=A + 128), "ALIGN"), (dict(batch=0), "OK"), (dict(T=0), "OK")]:
        assert chunk(L, **kw) == err(e), kw
    assert L.q8_attn_chunk_workspace_size(8, 3, 128) == 0
    assert L.q8_attn_chunk_workspace_size(8, 2, 96) == 0
    assert L.q8_attn_chunk_workspace_size(8, 2, 128) > 0


def exact_turns(f):
    """f / (2 pi) modulo one, in units of 2^-64, as a whole number (60 digits)."""
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918")
    return int((Decimal(f) / two_pi * 2 ** 64).to_integral_value()) % 2 ** 64


def test_rope_turns_are_exact(L):
    from block_quantized_int8_gb300 import q8
    f = np.concatenate([[0.0, 1.0, -1.0, math.pi, 65536.0, -65536.0, 1e-9, -1e-9, 5e-324, 2.0 ** -70],
                        10000.0 ** (-np.arange(64) / 64.0), np.random.default_rng(0).uniform(-1000, 1000, 200)])
    got = q8.rope_turns(f.tolist(), device="cpu").numpy().view(np.uint64)
    for x, t in zip(f, got):
        off = (int(t) - exact_turns(float(x))) % 2 ** 64
        # five rounded terms of half a unit each, and the exact value's
        assert min(off, 2 ** 64 - off) <= 3, (x, off)
    for bad in (math.nan, math.inf, 65537.0, -65537.0):
        with pytest.raises(q8.Q8Error):
            q8.rope_turns([1.0, bad], device="cpu")
    with pytest.raises(ValueError):
        q8.rope_turns([[1.0]], device="cpu")


def test_rope_frequencies():
    from block_quantized_int8_gb300 import q8
    f, m = q8.rope_frequencies(8, 10000.0)
    assert m == 1.0 and np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-14)
    g, m = q8.rope_frequencies(8, 10000.0, "linear", 4.0)
    assert m == 1.0 and np.allclose(g, np.array(f) / 4, rtol=1e-14)
    g, m = q8.rope_frequencies(8, 10000.0, "ntk", 4.0)
    assert m == 1.0 and g[0] == 1.0 and math.isclose(g[3], f[3] / 4, rel_tol=1e-12)
    f, _ = q8.rope_frequencies(128)
    g, m = q8.rope_frequencies(128, scaling="yarn", factor=16.0)
    assert math.isclose(m, 1 + 0.1 * math.log(16)) and g[0] == f[0] and math.isclose(g[-1], f[-1] / 16, rel_tol=1e-12)
    turns = [4096 * x / (2 * math.pi) for x in f]
    for a, b, n in zip(g, f, turns):
        assert b / 16 <= a * (1 + 1e-12) and a <= b
        if n > 33:
            assert a == b or n < 45  # the ramp begins at a whole pair
        if n < 0.8:
            assert math.isclose(a, b / 16, rel_tol=1e-12)
    for bad in (dict(rot=3), dict(rot=2), dict(rot=8, scaling="other"), dict(rot=8, factor=0.5), dict(rot=8, factor=math.nan)):
        with pytest.raises(ValueError):
            q8.rope_frequencies(**bad)
