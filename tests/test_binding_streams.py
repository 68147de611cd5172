"""What the binding allocates (outputs, zeroed workspaces) is allocated on the stream that the
call is given.  Runs without a GPU: the library and the streams are fakes."""
import types

import pytest
import torch

STREAM = 77


@pytest.fixture
def q8(monkeypatch):
    from block_quantized_int8_gb300 import q8

    class Lib:
        """Every size is 256, every call succeeds on the stream that its last argument names."""
        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_size_ex"):
                return lambda *a: 256

            def call(*a):
                assert a[-1] == STREAM
                seen.calls += 1
                return 0
            return call
    seen = types.SimpleNamespace(inside=0, made=[], calls=0)

    def new(stream, make):
        assert stream == STREAM
        seen.inside += 1
        try:
            return make()
        finally:
            seen.inside -= 1

    def recorded(make):
        def f(*a, **kw):
            seen.made.append(seen.inside)
            kw.pop("device", None)
            return make(*a, **kw)
        return f
    monkeypatch.setattr(q8, "_lib", Lib())
    monkeypatch.setattr(q8, "_new", new)
    monkeypatch.setattr(q8, "_cuda", lambda t, *a, **kw: t)
    fake = types.SimpleNamespace(**{n: getattr(torch, n) for n in ("float32", "float16", "bfloat16", "uint8", "int8", "Tensor")},
                                 empty=recorded(torch.empty), zeros=recorded(torch.zeros),
                                 cuda=types.SimpleNamespace(Stream=torch.cuda.Stream))
    monkeypatch.setattr(q8, "torch", fake)
    q8.seen = seen
    yield q8
    del q8.seen


def planes(n, k):
    return torch.zeros((n, k), dtype=torch.int8), torch.zeros((n, k // 32), dtype=torch.float16)


def x(m, k):
    return torch.zeros((m, k), dtype=torch.bfloat16)


CALLS = {
    "quantize_rows": (2, lambda q8: q8.q8_quantize_rows(torch.zeros(4, 64), stream=STREAM)),
    "gguf_to_planar": (2, lambda q8: q8.q8_gguf_to_planar(torch.zeros(4 * 2 * 34, dtype=torch.uint8), 4, 64, stream=STREAM)),
    "planar_to_gguf": (1, lambda q8: q8.q8_planar_to_gguf(*planes(4, 64), stream=STREAM)),
    "gemv": (2, lambda q8: q8.q8_gemv(*planes(4, 64), x(1, 64), stream=STREAM)),
    "gemm_skinny": (2, lambda q8: q8.q8_gemm_skinny(*planes(4, 64), x(3, 64), stream=STREAM)),
    "gemm_skinny_noalloc": (1, lambda q8: q8.q8_gemm_skinny_noalloc(*planes(4, 64), x(3, 64), stream=STREAM)),
    "linear_batch": (1, lambda q8: q8.q8_linear_batch([(*planes(4, 64), x(3, 64), torch.zeros(3, 4))], stream=STREAM)),
    "linear_chain": (1, lambda q8: q8.q8_linear_chain(*q8.make_chain([(*planes(4, 64), x(3, 64), torch.zeros(3, 4), 0)]), stream=STREAM)),
    "gemm_w8a8": (2, lambda q8: q8.q8_gemm_w8a8(*planes(4, 64), x(40, 64), stream=STREAM)),
    "gemm": (1, lambda q8: q8.q8_gemm(*planes(8, 64), x(40, 64), stream=STREAM)),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_made_on_the_given_stream(q8, name):
    count, call = CALLS[name]
    call(q8)
    assert q8.seen.calls == 1 and q8.seen.made == [1] * count
