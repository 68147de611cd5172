"""The binding of the prompt-step calls refuses what does not fit before the library is reached
(without a GPU: tensors that say they are on one, and a fake of the library)."""
import pytest
import torch

from test_binding_refusals import b16, f32, gpu, ints, planes, q8  # noqa: F401


def parts(q8):
    cache = q8.KvCache(*(t for pair in (planes(16, 64, (2, 1)), planes(16, 64, (2, 1))) for t in pair))
    turns = ints(32, dtype=torch.int64)
    ws = gpu(torch.zeros(256, dtype=torch.uint8))
    return {
        "norm": (q8.q8_rms_norm, dict(x=f32(3, 64), weight=f32(64), residual=b16(3, 64), residual_out=b16(3, 64), y=b16(3, 64),
                                      q=ints(3, 64, dtype=torch.int8), s=gpu(torch.zeros((3, 2), dtype=torch.float16)), dev_status=ints(1))),
        "rope": (q8.q8_rope, dict(x=b16(3, 2, 64), positions=ints(3), turns=turns, y=b16(3, 2, 64))),
        "append": (q8.q8_rope_append, dict(q=f32(3, 2, 64), k=f32(3, 1, 64), v=f32(3, 1, 64), cache=cache, positions=ints(3),
                                           slots=ints(3, dtype=torch.int64), turns=turns, y=b16(3, 2, 64), dev_status=ints(1))),
        "plan": (q8.q8_kv_plan, dict(table=ints(2, 4), lens=ints(2), new_tokens=ints(2), page_size=16, pages=8, T=5, free_pages=ints(6),
                                     free_count=ints(1), free_left=ints(1), starts=ints(3), slots=ints(5, dtype=torch.int64),
                                     positions=ints(5), lens_out=ints(2), dev_status=ints(1))),
        "chunk": (q8.q8_attn_chunk, dict(q=b16(5, 2, 64), cache=cache, table=ints(2, 4), lens=ints(2), starts=ints(3), out=b16(5, 2, 64),
                                         lse=f32(5, 2), ws=ws, dev_status=ints(1))),
    }


NAMES = ["norm", "rope", "append", "plan", "chunk"]


def call(q8, name, **kw):
    fn, args = parts(q8)[name]
    args.update(kw)
    return fn(**args, stream=0)


@pytest.mark.parametrize("name", NAMES)
def test_the_calls_are_reached_where_all_is_well(q8, name):  # noqa: F811
    with pytest.raises(AssertionError, match="was reached"):
        call(q8, name)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_the_host_are_refused(q8, name):  # noqa: F811
    for key, t in parts(q8)[name][1].items():
        if isinstance(t, torch.Tensor):
            with pytest.raises((TypeError, ValueError)):
                call(q8, name, **{key: t.as_subclass(torch.Tensor)})


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_type_are_refused(q8, name):  # noqa: F811
    for key, t in parts(q8)[name][1].items():
        if isinstance(t, torch.Tensor) and key != "ws":
            with pytest.raises((TypeError, ValueError)):
                call(q8, name, **{key: gpu(torch.zeros(t.shape, dtype=torch.float64))})


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_shape_are_refused(q8, name):  # noqa: F811
    for key, t in parts(q8)[name][1].items():
        # (a status word may be part of a longer array, the free list is as long as it is, x and q set the shape)
        if isinstance(t, torch.Tensor) and key not in ("ws", "dev_status", "free_pages"):
            bad = tuple(n + 1 if i == 0 else n for i, n in enumerate(t.shape))
            with pytest.raises((TypeError, ValueError)):
                call(q8, name, **{key: gpu(torch.zeros(bad, dtype=t.dtype))})


@pytest.mark.parametrize("name", NAMES)
def test_strides_that_do_not_fit_are_refused(q8, name):  # noqa: F811
    for key, t in parts(q8)[name][1].items():
        if isinstance(t, torch.Tensor) and key not in ("ws", "dev_status") and t.shape[-1] > 1:
            wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2]
            with pytest.raises((TypeError, ValueError)):
                call(q8, name, **{key: gpu(wide)})


def test_tensors_of_two_devices_are_refused(q8):  # noqa: F811
    class Other(type(f32(1))):
        def get_device(self):
            return 1
    for name in NAMES:
        for key, t in parts(q8)[name][1].items():
            if isinstance(t, torch.Tensor) and key not in ("dev_status", "x", "q", "table"):
                with pytest.raises(ValueError, match="device"):
                    call(q8, name, **{key: t.as_subclass(Other)})


def test_arguments_that_belong_together(q8):  # noqa: F811
    with pytest.raises(ValueError):
        call(q8, "norm", residual=None)
    with pytest.raises(ValueError):
        call(q8, "plan", free_pages=None)
    with pytest.raises(ValueError):
        call(q8, "plan", free_count=None)


def test_a_status_word_of_another_device_is_refused(q8):  # noqa: F811
    """Kernels write to it."""
    class Other(type(ints(1))):
        def get_device(self):
            return 1
    for name in ("norm", "append", "plan", "chunk"):
        with pytest.raises(ValueError, match="device"):
            call(q8, name, dev_status=ints(1).as_subclass(Other))


@pytest.mark.parametrize("B,width", [(0, 4), (2, 0), (2, 4)])
def test_an_empty_free_list_is_a_list(q8, monkeypatch, B, width):  # noqa: F811
    """Its tensor has no address, nor has an empty table: the library gets another, as NULL is no list (free_left is then not written)."""
    class Empty(type(ints(1))):
        def data_ptr(self):
            return 0 if self.numel() == 0 else 1 << 20
    given = []
    monkeypatch.setattr(q8.lib(), "q8_kv_plan", lambda *a: given.append(a) or 0, raising=False)
    call(q8, "plan", table=ints(B, width).as_subclass(Empty), lens=ints(B), new_tokens=ints(B), starts=ints(B + 1), lens_out=ints(B),
         free_pages=ints(0).as_subclass(Empty))
    assert given[0][7] and given[0][8] == 0
