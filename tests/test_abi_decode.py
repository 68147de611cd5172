"""The decode-step entry points refuse bad arguments on the host, before any
CUDA call (so these run without a GPU)."""
import ctypes
import math

import pytest

A = 1 << 20  # a well-aligned fake device address, never touched


@pytest.fixture(scope="module")
def L():
    from block_quantized_int8_gb300 import build, q8
    build.build()
    return q8.lib()


def cache(**kw):
    from block_quantized_int8_gb300 import q8
    d = dict(kq=A, ks=A, vq=A, vs=A, pages=4, page_size=16, kv_heads=2, head_dim=128)
    d.update(kw)
    return q8._CKvCache(*(d[n] for n, _ in q8._CKvCache._fields_))


BAD_CACHES = [(dict(page_size=8), "SHAPE"), (dict(page_size=24), "SHAPE"), (dict(page_size=2048), "SHAPE"),
              (dict(head_dim=96), "SHAPE"), (dict(kv_heads=0), "SHAPE"), (dict(pages=0), "SHAPE"),
              (dict(kq=None), "ARG"), (dict(vs=None), "ARG"), (dict(ks=A + 8), "ALIGN"), (dict(vq=A + 4), "ALIGN")]


def rows(L, fn, c=None, k=A, v=A, ldk=256, ldv=256, dtype=0, slots=A, T=3, status=None):
    c = cache() if c is None else c
    ref = ctypes.byref(c) if c else None
    if fn == "append":
        return L.q8_kv_append(ref, k, v, ldk, ldv, dtype, slots, T, status, None)
    return L.q8_kv_read(ref, slots, T, k, v, ldk, ldv, dtype, status, None)


@pytest.mark.parametrize("fn", ["append", "read"])
def test_kv_rows_validation(L, fn):
    from block_quantized_int8_gb300 import q8
    for kw, err in BAD_CACHES:
        assert rows(L, fn, cache(**kw)) == getattr(q8, "Q8_ERR_" + err), kw
    assert rows(L, fn, c=False) == q8.Q8_ERR_ARG
    assert rows(L, fn, dtype=2) == q8.Q8_ERR_ARG
    assert rows(L, fn, T=-1) == q8.Q8_ERR_SHAPE
    assert rows(L, fn, ldk=255) == q8.Q8_ERR_SHAPE
    assert rows(L, fn, ldv=0) == q8.Q8_ERR_SHAPE
    assert rows(L, fn, ldk=258) == q8.Q8_ERR_ALIGN
    assert rows(L, fn, ldk=260, dtype=1) == q8.Q8_ERR_ALIGN
    for a in ("k", "v", "slots"):
        assert rows(L, fn, **{a: None}) == q8.Q8_ERR_ARG
        assert rows(L, fn, **{a: A + 4}) == q8.Q8_ERR_ALIGN
    assert rows(L, fn, status=A + 2) == q8.Q8_ERR_ALIGN
    assert rows(L, fn, T=0) == q8.Q8_OK


def attn(L, c=None, q=A, ldq=1024, heads=8, table=A, width=4, lens=A, batch=3, scale=0.1, cap=0.0, window=0, out=A, lse=A,
         ws=A, wsb=1 << 40, status=None):
    c = cache() if c is None else c
    return L.q8_attn_decode(ctypes.byref(c) if c else None, q, ldq, heads, table, width, lens, batch, scale, cap, window, out,
                            lse, ws, wsb, status, None)


def test_attn_validation(L):
    from block_quantized_int8_gb300 import q8
    for kw, err in BAD_CACHES:
        assert attn(L, cache(**kw)) == getattr(q8, "Q8_ERR_" + err), kw
    assert attn(L, c=False) == q8.Q8_ERR_ARG
    assert attn(L, heads=7) == q8.Q8_ERR_SHAPE       # not a multiple of the key heads
    assert attn(L, heads=0) == q8.Q8_ERR_SHAPE
    assert attn(L, batch=-1) == q8.Q8_ERR_SHAPE
    assert attn(L, ldq=1023) == q8.Q8_ERR_SHAPE
    assert attn(L, ldq=1028) == q8.Q8_ERR_ALIGN
    assert attn(L, width=-1) == q8.Q8_ERR_SHAPE
    assert attn(L, width=1 << 28) == q8.Q8_ERR_SHAPE  # 2^32 tokens
    assert attn(L, window=-1) == q8.Q8_ERR_ARG
    assert attn(L, cap=-1.0) == q8.Q8_ERR_ARG
    for bad in (math.nan, math.inf):
        assert attn(L, scale=bad) == q8.Q8_ERR_ARG
        assert attn(L, cap=bad) == q8.Q8_ERR_ARG
    for a in ("q", "table", "lens", "out"):
        assert attn(L, **{a: None}) == q8.Q8_ERR_ARG
    for a, off in (("q", 8), ("table", 2), ("lens", 2), ("out", 8), ("lse", 2), ("status", 2), ("ws", 128)):
        assert attn(L, **{a: A + off}) == q8.Q8_ERR_ALIGN, a
    need = L.q8_attn_decode_workspace_size(3, 8, 2, 128)
    assert need > 0
    assert attn(L, ws=None) == q8.Q8_ERR_WORKSPACE
    assert attn(L, wsb=need - 1) == q8.Q8_ERR_WORKSPACE
    assert attn(L, batch=0) == q8.Q8_OK
    assert L.q8_attn_decode_workspace_size(3, 7, 2, 128) == 0
    assert L.q8_attn_decode_workspace_size(3, 8, 2, 96) == 0
    assert L.q8_attn_decode_workspace_size(0, 8, 2, 128) == 0


def moe(L, x=A, ldx=64, logits=A, ldl=8, T=3, E=8, k=2, q13=A, s13=A, q2=A, s2=A, H=64, F=96, y=A, ldy=64, ids=A, w=A, ws=A,
        wsb=1 << 40, status=None):
    return L.q8_moe(x, ldx, logits, ldl, T, E, k, 1, q13, s13, q2, s2, H, F, y, ldy, ids, w, ws, wsb, status, None)


def test_moe_validation(L):
    from block_quantized_int8_gb300 import q8
    for kw in (dict(T=-1), dict(T=33), dict(E=0), dict(E=513), dict(H=48), dict(F=0), dict(H=0), dict(F=33), dict(ldx=63),
               dict(ldl=7), dict(ldy=63), dict(H=8224, ldx=8224, ldy=8224), dict(F=65568)):
        assert moe(L, **kw) == q8.Q8_ERR_SHAPE, kw
    for kw in (dict(k=0), dict(k=9), dict(k=17, E=32, ldl=32)):
        assert moe(L, **kw) == q8.Q8_ERR_ARG, kw
    for a in ("x", "logits", "q13", "s13", "q2", "s2", "y"):
        assert moe(L, **{a: None}) == q8.Q8_ERR_ARG, a
    for a, off in (("x", 8), ("logits", 2), ("q13", 8), ("s13", 2), ("q2", 4), ("s2", 8), ("y", 2), ("ids", 1), ("w", 2),
                   ("ws", 16), ("status", 1)):
        assert moe(L, **{a: A + off}) == q8.Q8_ERR_ALIGN, a
    assert moe(L, ldx=68) == q8.Q8_ERR_ALIGN
    need = L.q8_moe_workspace_size(3, 8, 64, 96, 2)
    assert need > 0
    assert moe(L, ws=None) == q8.Q8_ERR_WORKSPACE
    assert moe(L, wsb=need - 1) == q8.Q8_ERR_WORKSPACE
    assert moe(L, T=0) == q8.Q8_OK
    assert L.q8_moe_workspace_size(33, 8, 64, 96, 2) == 0
    assert L.q8_moe_workspace_size(3, 8, 64, 96, 9) == 0


def sample(L, logits=A, dtype=0, ld=100, rows=2, V=100, T=A, k=A, p=A, m=A, u=A, tok=A, lp=A, kept=A, status=None):
    return L.q8_sample(logits, dtype, ld, rows, V, T, k, p, m, u, tok, lp, kept, status, None)


def test_sample_validation(L):
    from block_quantized_int8_gb300 import q8
    assert sample(L, dtype=2) == q8.Q8_ERR_ARG
    for kw in (dict(V=0), dict(V=(1 << 19) + 1, ld=1 << 21), dict(ld=99), dict(rows=-1)):
        assert sample(L, **kw) == q8.Q8_ERR_SHAPE, kw
    for a in ("logits", "u", "tok"):
        assert sample(L, **{a: None}) == q8.Q8_ERR_ARG, a
    for a in ("logits", "T", "k", "p", "m", "u", "tok", "lp", "kept", "status"):
        assert sample(L, **{a: A + 2}) == q8.Q8_ERR_ALIGN, a
    assert sample(L, logits=A + 1, dtype=1) == q8.Q8_ERR_ALIGN
    assert sample(L, rows=0) == q8.Q8_OK
