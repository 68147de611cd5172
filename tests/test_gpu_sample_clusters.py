"""q8_sample with fewer CTAs a row than a whole GPU runs (as on a part of one): the same draws,
or Q8_ERR_UNSUPPORTED where a row's slices find no room."""
import numpy as np
import pytest
import torch

import test_gpu_sample as sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [1, 2, 4, 8])
@pytest.mark.parametrize("V", [3000, 50000, 100003, 204000, 400000])
@pytest.mark.parametrize("bf16", [False, True])
def test_fewer_ctas_a_row(monkeypatch, most, V, bf16):
    from block_quantized_int8_gb300 import q8
    l, u, r = sample.rows(5, V, V)
    logits = torch.from_numpy(l).cuda()
    logits = logits.to(torch.bfloat16) if bf16 else logits
    knobs = dict(T=[1.0, 0.7, 2.0, 0.0, 1.0], k=[0, 50, 2000, 0, 0], p=[0.95, 0.9, 0.99, 1.0, 1.0])
    want = sample.draw(logits, u, **knobs)
    monkeypatch.setenv("Q8_SAMPLE_CLUSTER", str(most))
    if V > most * 51000:  # a slice is at most 226 KB less 26 of lists and counts
        with pytest.raises(q8.Q8Error) as e:
            sample.draw(logits, u, **knobs)
        assert e.value.status == q8.Q8_ERR_UNSUPPORTED
    else:
        assert all(np.array_equal(a, b) for a, b in zip(sample.draw(logits, u, **knobs), want))
