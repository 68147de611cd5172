"""The cases of perf/more_operators.py: the library's calls give what the plain forms give when a state's frequencies or its
cache's tensors change after a first pass, in place or for others."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def both(m, state):
    """(plain form's outputs, library's) of one state."""
    out = []
    for m.own in (False, True):
        out.append([t.clone() for t in m.run(state)])
    return out


def near(a, b):
    """Within a bf16 rounding, and for the cache's values a code, of the largest value."""
    for x, y in zip(a, b):
        assert float((x.float() - y.float()).abs().max()) <= (2.0 ** -7 + 1 / 127) * float(x.float().abs().max())


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", ["rope_5", "rope_append_1"])
def test_frequencies_that_change(name, in_place):
    from perf import more_operators as m
    case = next(c for c in m.listed() if c["name"] == name)
    st = m.prepare(case, 1)
    near(*both(m, st))
    first = both(m, st)[1]
    if in_place:
        st["inv_freq"].mul_(0.37)
    else:
        st["inv_freq"] = st["inv_freq"] * 0.37
    plain, own = both(m, st)
    near(plain, own)
    assert not torch.equal(first[0], own[0])


def replace_planes(st):
    for k in ("kq", "ks", "vq", "vs"):
        old = st[k]
        st[k] = old.roll(1, 0).clone()
        old.zero_()


def test_cache_tensors_that_are_replaced_are_read():
    from perf import more_operators as m
    st = m.prepare(next(c for c in m.listed() if c["name"] == "chunk_16x5"), 1)
    both(m, st)
    replace_planes(st)
    plain, own = both(m, st)
    near(plain, own)


def test_cache_tensors_that_are_replaced_are_written():
    from perf import more_operators as m
    st = m.prepare(next(c for c in m.listed() if c["name"] == "rope_append_1"), 1)
    both(m, st)
    replace_planes(st)
    m.own = True
    for k in ("kq", "vq"):
        st[k].zero_()
    m.run(st)
    assert bool((st["kq"] != 0).any()) and bool((st["vq"] != 0).any())
