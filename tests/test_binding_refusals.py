"""A tensor that is not on the GPU never reaches a kernel: the binding refuses it, the status word
and the workspace among them.  Runs without a GPU (a fake of the library fails the test if it is
called)."""

import pytest
import torch


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU, and gives an address that nobody reads."""
    is_cuda = True

    def data_ptr(self):
        return 1 << 20


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def q8(monkeypatch):
    from block_quantized_int8_gb300 import q8

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_size_ex"):
                return lambda *a: 256

            def call(*a):
                raise AssertionError(f"{name} was reached")
            return call
    monkeypatch.setattr(q8, "_lib", Lib())
    return q8


def planes(n, k, lead=()):
    return gpu(torch.zeros((*lead, n, k), dtype=torch.int8)), gpu(torch.zeros((*lead, n, k // 32), dtype=torch.float16))


def f32(*shape):
    return gpu(torch.zeros(shape))


def b16(*shape):
    return gpu(torch.zeros(shape, dtype=torch.bfloat16))


def ints(*shape, dtype=torch.int32):
    return gpu(torch.zeros(shape, dtype=dtype))


def calls(q8):
    cache = q8.KvCache(*(t for pair in (planes(16, 64, (2, 1)), planes(16, 64, (2, 1))) for t in pair))
    ws = gpu(torch.zeros(256, dtype=torch.uint8))
    attn = dict(out=b16(1, 2, 64), lse=f32(1, 2))
    moe = (b16(1, 64), f32(1, 2), *planes(128, 64, (2,)), *planes(64, 64, (2,)), 1)
    moe_out = dict(y=f32(1, 64), ids=ints(1, 1), weights=f32(1, 1))
    skinny = (*planes(8, 64), b16(3, 64))
    return {
        "quantize": lambda **kw: q8.q8_quantize_rows(f32(2, 64), *planes(2, 64), stream=0, **kw),
        "gemv": lambda **kw: q8.q8_gemv(*planes(8, 64), b16(64), y=f32(8), stream=0, **kw),
        "skinny": lambda **kw: q8.q8_gemm_skinny(*skinny, y=f32(3, 8), stream=0, **kw),
        "batch": lambda **kw: q8.q8_linear_batch([(*skinny, f32(3, 8))], stream=0, **kw),
        "chain": lambda **kw: q8.q8_linear_chain(*q8.make_chain([(*skinny, f32(3, 8), 0)]), stream=0, **kw),
        "w8a8": lambda **kw: q8.q8_gemm_w8a8(*skinny, y=f32(3, 8), stream=0, **kw),
        "gemm": lambda **kw: q8.q8_gemm(*planes(8, 64), b16(40, 64), y=b16(40, 8), stream=0, **kw),
        "append": lambda **kw: q8.q8_kv_append(cache, f32(1, 64), f32(1, 64), ints(1, dtype=torch.int64), stream=0, **kw),
        "read": lambda **kw: q8.q8_kv_read(cache, ints(1, dtype=torch.int64), f32(1, 64), f32(1, 64), stream=0, **kw),
        "attn": lambda ws=ws, **kw: q8.q8_attn_decode(b16(1, 2, 64), cache, ints(1, 2), ints(1), **attn, ws=ws, stream=0, **kw),
        "moe": lambda ws=ws, **kw: q8.q8_moe(*moe, **moe_out, ws=ws, stream=0, **kw),
        "sample": lambda **kw: q8.q8_sample(f32(1, 40), f32(1), token=ints(1), logprob=f32(1), kept=ints(1), stream=0, **kw),
    }


NAMES = ["quantize", "gemv", "skinny", "batch", "chain", "w8a8", "gemm", "append", "read", "attn", "moe", "sample"]


@pytest.mark.parametrize("name", NAMES)
def test_a_status_word_on_the_host_is_refused(q8, name):
    with pytest.raises(TypeError, match="dev_status"):
        workspaces = {"ws": gpu(torch.zeros(256, dtype=torch.uint8))} if name in ("gemv", "skinny", "batch", "chain", "w8a8") else {}
        calls(q8)[name](dev_status=torch.zeros(1, dtype=torch.int32), **workspaces)


@pytest.mark.parametrize("name", ["append", "attn", "moe", "sample"])
@pytest.mark.parametrize("bad", [torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32)])
def test_a_status_of_another_width_or_none_is_refused(q8, name, bad):
    with pytest.raises(TypeError, match="dev_status"):
        calls(q8)[name](dev_status=gpu(bad))


@pytest.mark.parametrize("name", ["gemv", "skinny", "batch", "chain", "w8a8", "attn", "moe"])
def test_a_workspace_on_the_host_is_refused(q8, name):
    with pytest.raises(TypeError, match="ws"):
        calls(q8)[name](ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="ws"):
        calls(q8)[name](ws=gpu(torch.zeros(512, dtype=torch.uint8))[::2])


@pytest.mark.parametrize("which", ["gemv", "w8a8", "gemm"])
@pytest.mark.parametrize("at", ["q", "s", "x", "y"])
def test_operands_on_the_host_are_refused(q8, which, at):
    m = {"gemv": 1, "w8a8": 3, "gemm": 40}[which]
    a = dict(zip("qs", planes(8, 64)), x=b16(64) if which == "gemv" else b16(m, 64),
             y=f32(8) if which == "gemv" else (f32(m, 8) if which == "w8a8" else b16(m, 8)))
    a[at] = a[at].as_subclass(torch.Tensor)
    fn = {"gemv": q8.q8_gemv, "w8a8": q8.q8_gemm_w8a8, "gemm": q8.q8_gemm}[which]
    with pytest.raises(TypeError, match=at):
        fn(a["q"], a["s"], a["x"], y=a["y"], stream=0)


def test_the_calls_are_reached_where_all_is_well(q8):
    for name in NAMES:
        with pytest.raises(AssertionError, match="was reached"):
            workspaces = {"ws": gpu(torch.zeros(256, dtype=torch.uint8))} if name in ("gemv", "skinny", "batch", "chain", "w8a8") else {}
            calls(q8)[name](dev_status=ints(1), **workspaces)
