"""q8_rms_norm against its definition in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, half a step of binary32): h has one rounding (u); the
sum of squares has, in any order used here, chains of at most 42 additions (32 in a thread, 10 over
threads), so it is within 44 u of its value and its root's reciprocal within 22 u + 2 of the
reciprocal square root's own steps; three products follow.  Together below 2^-18 of y, to which h's
rounding adds u of |h| times the same factors.  bf16 rounds by 2^-8 of the value at most.  A Q8_0
value is off by half a scale, the scale itself by 2^-11 (2^-25 below the normal range) and what
y is off.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FINE = 2.0 ** -18


def definition(x, res, w, offset, eps):
    h = x.astype(np.float64) + (0.0 if res is None else res.astype(np.float64))
    f = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    g = 1.0 if w is None else w.astype(np.float64) + offset
    return h, h * f * g, np.abs(f * g) * np.ones_like(h)


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def run(x, res=None, w=None, offset=0.0, eps=1e-6, in_place=True, quantized=True, bf16=True, status=0):
    from block_quantized_int8_gb300 import q8
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, rd = x.cuda(), None if res is None else res.cuda()
    ro = None if res is None or in_place else torch.full_like(rd, 7.0)
    y, q, s = q8.q8_rms_norm(xd, None if w is None else w.cuda(), offset, eps, rd, ro, quantized=quantized, bf16=bf16, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    h, ref, gain = definition(f64(x), None if res is None else f64(res), None if w is None else f64(w), offset, eps)
    slack = FINE * np.abs(ref) + 2.0 ** -24 * np.abs(h) * gain + 1e-37
    if res is not None:
        got = f64(rd if in_place else ro)
        step = 2.0 ** -24 + (2.0 ** -8 if res.dtype == torch.bfloat16 else 0.0)
        assert np.all(np.abs(got - h) <= step * np.abs(h) * 1.01 + 1e-37)
        if not in_place:
            assert torch.equal(rd.cpu(), res)
    assert torch.equal(xd.cpu(), x)
    if bf16:
        assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + slack)
    else:
        assert y is None
    if quantized:
        sv = f64(s)
        top = np.abs(ref).reshape(*ref.shape[:-1], -1, 32).max(-1)
        assert np.all(np.abs(sv - top / 127) <= (2.0 ** -11 + 2 * FINE) * top / 127 + 2.0 ** -25)
        v = f64(q) * np.repeat(sv, 32, -1)
        # a scale rounded down leaves its largest value up to 2^-11 of 127 scales beyond the last code
        assert np.all(np.abs(v - ref) <= (0.5 + 127 * 2.0 ** -11) * np.repeat(sv, 32, -1) + slack + 127 * 2.0 ** -25)
    return y, q, s


def rows(n, w, seed, kind=torch.float32, spread=1.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, w)) * spread
    x[:, 3] *= 30
    return torch.from_numpy(x.astype(np.float32)).to(kind)


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("n,w", [(1, 32), (1, 1536), (3, 64), (5, 96), (2, 1024), (7, 2048), (4, 2080), (3, 5120), (2, 8192),
                                 (2, 8224), (1, 16384), (2, 32736), (1, 32768), (513, 416)])
@pytest.mark.parametrize("xk,rk", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16), (F32, None), (BF16, None)])
def test_widths_and_types(n, w, xk, rk):
    gain = rows(1, w, 9)[0] * 0.2 + 1
    run(rows(n, w, 1, xk), None if rk is None else rows(n, w, 2, rk, 3.0), gain, in_place=(n + w) % 2 == 0)


@pytest.mark.parametrize("offset", [0.0, 1.0, -0.5])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-2])
def test_gains_offsets_and_eps(offset, eps):
    run(rows(3, 256, 3), None, rows(1, 256, 4)[0] * 0.1, offset, eps)
    run(rows(3, 256, 5), rows(3, 256, 6), None, 0.0, eps)


@pytest.mark.parametrize("kind", [F32, BF16])
def test_strides_and_given_outputs(kind):
    from block_quantized_int8_gb300 import q8
    big = rows(5, 3 * 128, 7, kind).cuda()
    x, r = big[:, 128:256], big[:, 256:].clone()
    y = torch.full((5, 256), 9.0, dtype=BF16, device="cuda")
    out, q, s = q8.q8_rms_norm(x, residual=r, y=y[:, 64:192])
    assert q is None and s is None and out.data_ptr() == y[:, 64:192].data_ptr()
    h, ref, gain = definition(f64(big[:, 128:256]), f64(big[:, 256:]), None, 0.0, 1e-6)
    assert np.all(np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + FINE * np.abs(ref) + 2.0 ** -24 * np.abs(h) * gain)
    assert torch.all(y[:, :64] == 9.0) and torch.all(y[:, 192:] == 9.0)


def test_outputs_one_at_a_time_are_the_same():
    from block_quantized_int8_gb300 import q8
    x, r = rows(6, 640, 8, BF16).cuda(), rows(6, 640, 9).cuda()
    y, q, s = q8.q8_rms_norm(x, residual=r.clone(), quantized=True)
    y1, q1, _ = q8.q8_rms_norm(x, residual=r.clone())
    y2, q2, s2 = q8.q8_rms_norm(x, residual=r.clone(), bf16=False, quantized=True)
    assert q1 is None and y2 is None
    assert torch.equal(y, y1) and torch.equal(q, q2) and torch.equal(s, s2)
    # in place of x
    x2 = x.clone()
    q8.q8_rms_norm(x2, residual=r.clone(), y=x2)
    assert torch.equal(x2, y)


def test_a_row_onto_itself():
    from block_quantized_int8_gb300 import q8
    x = rows(5, 320, 20).cuda()
    y, _, _ = q8.q8_rms_norm(x.clone(), residual=x.clone())
    z = x.clone()
    y2, _, _ = q8.q8_rms_norm(z, residual=z)
    assert torch.equal(y, y2) and torch.equal(z, x + x)


def test_the_residual_may_go_to_x():
    from block_quantized_int8_gb300 import q8
    x, r = rows(6, 640, 8).cuda(), rows(6, 640, 9).cuda()
    y, _, _ = q8.q8_rms_norm(x.clone(), residual=r.clone())
    x2 = x.clone()
    y2, _, _ = q8.q8_rms_norm(x2, residual=r, residual_out=x2)
    assert torch.equal(y, y2) and torch.equal(x2, x + r)


@pytest.mark.parametrize("spread", [1e-40, 1e-30, 1e-20, 1e-12, 1e15, 1e19, 1e30, 1e36])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-38])
def test_rows_at_the_ends_of_the_range(spread, eps):
    x = rows(3, 512, 10, F32, spread)
    if spread == 1e-40:
        # subnormals: their own steps are 2^-149; the norm of what is there is still a norm
        x[0] = 0.0
    from block_quantized_int8_gb300 import q8
    y, _, _ = q8.q8_rms_norm(x.cuda(), eps=eps)
    with np.errstate(divide="ignore", invalid="ignore"):
        _, ref, _ = definition(f64(x), None, None, 0.0, eps if eps != 1e-6 else float(np.float32(1e-6)))
    ref = np.nan_to_num(ref) if eps == 0.0 else ref  # a row of zeros is zeros
    assert np.all(np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + 2.0 ** -17 * np.abs(ref) + 1e-38), np.abs(f64(y) - ref).max()


def test_rows_with_infinities_and_nan_stay_by_themselves():
    from block_quantized_int8_gb300 import q8
    x = rows(5, 256, 11)
    x[1, 40], x[3, 7] = np.inf, np.nan
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, q, s = q8.q8_rms_norm(x.cuda(), quantized=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == q8.Q8_DEV_NONFINITE
    y = f64(y)
    assert np.isnan(y[1, 40]) and np.all(y[1, :40] == 0) and np.all(y[1, 41:] == 0) and np.all(np.isnan(y[3]))
    _, ref, _ = definition(f64(x[[0, 2, 4]]), None, None, 0.0, 1e-6)
    assert np.all(np.abs(y[[0, 2, 4]] - ref) <= 2.0 ** -8 * np.abs(ref) * 1.01 + FINE * np.abs(ref))
    # the block that holds one is zeros
    assert torch.all(q[1, 32:64] == 0) and float(s[1, 1]) == 0.0 and torch.all(q[3] == 0)


def test_values_too_large_for_a_scale_are_flagged():
    from block_quantized_int8_gb300 import q8
    x, w = rows(2, 64, 12), torch.ones(64)
    w[40] = 1e9
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, q, s = q8.q8_rms_norm(x.cuda(), w.cuda(), quantized=True, dev_status=st)
    assert int(st.item()) == q8.Q8_DEV_SCALE_OVF and torch.all(q[:, 32:] == 0) and torch.all(s[:, 1] == 0) and torch.any(q[:, :32] != 0)


def test_the_codes_are_the_quantizers():
    """Where the gains make y exactly representable, codes and scales are those of q8_quantize_rows."""
    from block_quantized_int8_gb300 import q8
    r = np.random.default_rng(13)
    x = torch.from_numpy(np.where(r.random((9, 128)) < 0.5, -1.0, 1.0).astype(np.float32)).cuda()  # norm 1, eps 0: y = x w
    w = rows(1, 128, 14)[0].cuda()
    _, q, s = q8.q8_rms_norm(x, w, eps=0.0, bf16=False, quantized=True)
    q2, s2 = q8.q8_quantize_rows((x * w).contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_no_rows():
    from block_quantized_int8_gb300 import q8
    y, q, s = q8.q8_rms_norm(torch.empty((0, 64), device="cuda"), quantized=True)
    assert y.shape == (0, 64) and q.shape == (0, 64) and s.shape == (0, 2)
