"""The draw of the next token (q8_sample) against the binary64 definition: the
words kept, that the word drawn is the one whose share of the distribution
holds u, and its log-probability.  Binary32 exponentials are off by less than
2^-21, so shares by less than 2^-20; where a filter's edge falls within that, either
side counts (decode_ref.sample).  Cases with exact masses are checked exactly."""
import numpy as np
import pytest
import torch

import decode_ref as ref

pytestmark = pytest.mark.gpu


def draw(logits, u, T=None, k=None, p=None, m=None, status=0, stream=None):
    from block_quantized_int8_gb300 import q8
    n = logits.shape[0]

    def dev(a, t):
        return None if a is None else torch.from_numpy(np.broadcast_to(np.asarray(a, dtype=t), (n,)).copy()).cuda()
    lg = logits if isinstance(logits, torch.Tensor) else torch.from_numpy(logits).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dev(T, np.float32), dev(k, np.int32), dev(p, np.float32), dev(m, np.float32))
    uu = dev(u, np.float32)
    torch.cuda.synchronize()
    tok, lp, kept = q8.q8_sample(lg, uu, *args, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return tok.cpu().numpy(), lp.cpu().numpy(), kept.cpu().numpy()


def check(logits, u, T=1.0, k=0, p=1.0, m=0.0, **kw):
    n = logits.shape[0]
    tok, lp, kept = draw(logits, u, T, k, p, m, **kw)
    host = logits.float().cpu().numpy() if isinstance(logits, torch.Tensor) else logits
    b = [np.broadcast_to(np.asarray(a, dtype=t), (n,)) for a, t in ((T, np.float32), (k, np.int64), (p, np.float32), (m, np.float32), (u, np.float32))]
    for i in range(n):
        (lo, hi), prob, slack = ref.sample(host[i], float(b[0][i]), int(b[1][i]), float(b[2][i]), float(b[3][i]), float(b[4][i]))
        if hi == 0:
            assert tok[i] == -1 and lp[i] == -np.inf and kept[i] == 0
            continue
        assert lo <= kept[i] <= hi, (i, lo, kept[i], hi)
        t = tok[i]
        assert 0 <= t < host.shape[1] and prob[t] > 0, (i, t)
        c = np.cumsum(prob)
        assert c[t] - prob[t] - slack <= b[4][i] <= c[t] + slack, (i, t, c[t] - prob[t], b[4][i], c[t])
        want = np.log(prob[t])
        assert abs(lp[i] - want) <= (2.0 ** -19 + slack) * (1 + abs(want)), (i, lp[i], want)
    return tok, lp, kept


def rows(n, V, seed, sd=2.5):
    r = np.random.default_rng(seed)
    return (r.standard_normal((n, V)) * sd).astype(np.float32), r.random(n).astype(np.float32), r


@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4096, 4097, 32003, 131071, 262144])
def test_vocabularies(V):
    l, u, r = rows(6, V, V)
    check(l, u, T=[1.0, 0.7, 1.3, 1.0, 0.5, 2.0], k=[0, 50, 0, 7, 1, V], p=[1.0, 0.95, 0.9, 1.0, 0.3, 0.999],
          m=[0.0, 0.0, 0.05, 0.01, 0.0, 0.0])


def test_largest_vocabulary():
    l, u, r = rows(2, 1 << 19, 1)
    check(l, u, k=[0, 300], p=[0.9, 0.9])


@pytest.mark.parametrize("n", [1, 3, 64, 400])
def test_rows(n):
    l, u, r = rows(n, 5000, n)
    check(l, u, T=r.choice([0.0, 0.6, 1.0, 1.5], n), k=r.choice([0, 1, 20, 400, 6000], n), p=r.choice([0.1, 0.9, 1.0], n),
          m=r.choice([0.0, 0.1], n))


@pytest.mark.parametrize("n,V", [(153, 3001), (512, 700), (513, 700), (80, 20000)])
def test_rows_of_mixed_knobs_beyond_one_wave(n, V):
    # greedy rows, short and long lists, top-p alone and none, in any order
    l, u, r = rows(n, V, n + V, sd=4.0)
    kind = r.integers(0, 6, n)
    check(l, u, np.where(kind == 0, 0.0, 0.8), np.array([0, 20, 1500, 0, 0, 40])[kind],
          np.array([1.0, 1.0, 0.9, 0.95, 1.0, 0.5])[kind], np.where(kind == 4, 0.01, 0.0))


def test_defaults_are_the_plain_distribution():
    from block_quantized_int8_gb300 import q8
    l, u, r = rows(40, 700, 9)
    check(l, u)
    tok, lp, kept = draw(l, u)
    a = check(l, u, T=1.0, k=0, p=1.0, m=0.0)
    assert np.array_equal(tok, a[0]) and np.array_equal(lp, a[1]) and np.array_equal(kept, a[2])


def test_bf16_logits_and_their_ties():
    r = np.random.default_rng(4)
    x = torch.from_numpy((r.standard_normal((8, 50001)) * 2).astype(np.float32)).to(torch.bfloat16).cuda()
    check(x, r.random(8), k=[100, 500, 0, 0, 1000, 20, 3, 0], p=[1.0, 0.9, 0.8, 0.99, 0.7, 0.5, 1.0, 0.2])


def test_greedy_takes_the_first_of_the_largest():
    l = np.zeros((4, 9000), dtype=np.float32)
    l[0, [17, 8000]] = 3.0
    l[2, 8999] = 1e30
    l[3, :] = -5.0
    l[3, 0] = -np.inf
    tok, lp, kept = draw(l, [0.9, 0.9, 0.5, 0.99], T=[0.0, -1.0, 0.0, 0.0])
    assert tok.tolist() == [17, 0, 8999, 1] and np.all(lp == 0) and np.all(kept == 1)


def test_equal_logits_are_exact():
    # every word has the same mass: the token is floor(u * kept) of the first `kept`
    V = 20000
    l = np.full((6, V), -2.5, dtype=np.float32)
    u = np.array([0.0, 0.25, 0.5, 0.75, 0.9375, 0.125], dtype=np.float32)
    tok, lp, kept = draw(l, u, k=[0, 1000, 16, 0, 4096, 1], p=[1.0, 1.0, 0.5, 0.25, 0.75, 1.0])
    n = np.array([V, 1000, 8, V // 4, int(4096 * 0.75), 1])
    assert np.array_equal(kept, n)
    assert np.array_equal(tok, np.floor(u * n).astype(int))
    assert np.all(np.abs(lp + np.log(n)) <= 2.0 ** -20 * np.log(n))


def test_ties_at_the_last_place_go_to_the_lowest_indexes():
    l = np.full((3, 12000), -30.0, dtype=np.float32)
    l[:, [11, 5000, 6000, 11999]] = 1.0
    l[:, 9000] = 1.0
    tok, lp, kept = draw(l, [0.0, 0.5, 0.999], T=1.0, k=3)
    assert kept.tolist() == [3, 3, 3] and tok.tolist() == [11, 5000, 6000]
    tok, lp, kept = draw(l, [0.0, 0.5, 0.999], T=0.01, p=[0.59, 0.6, 0.61])
    # five equal shares: 0.6f is just above 3/5, so the fourth is kept from there on
    assert kept.tolist() == [3, 4, 4] and tok.tolist() == [11, 6000, 9000]


def test_forbidden_words_and_special_values():
    from block_quantized_int8_gb300 import q8
    l, u, r = rows(6, 3001, 12)
    l[0, :] = -np.inf                      # nothing left
    l[1, 1:] = -np.inf                     # one word
    l[2, :] = np.finfo(np.float32).min     # the type's lowest value everywhere
    l[3, 7] = np.inf
    l[4, ::2] = -np.inf
    l[5, 5] = np.finfo(np.float32).max
    check(l, u, T=0.9, k=[0, 5, 10, 0, 40, 0], p=[0.9, 0.9, 1.0, 0.9, 0.9, 1.0])
    l[4, 1] = np.nan
    check(l, u, T=0.9, k=[0, 5, 10, 0, 40, 0], p=0.9, status=q8.Q8_DEV_NONFINITE)
    tok, lp, kept = draw(l[3:5], u[:2], m=1.5, status=q8.Q8_DEV_NONFINITE)   # min-p above one leaves nothing
    assert tok.tolist() == [-1, -1] and kept.tolist() == [0, 0]


def test_edges_of_u_and_p():
    l, u, r = rows(4, 2000, 13)
    check(l, np.float32([0.0, 1.0 - 2.0 ** -24, 0.0, 1.0 - 2.0 ** -24]), p=[1.0, 1.0, 0.0, 1e-9])


def test_high_and_low_temperatures():
    l, u, r = rows(4, 30000, 14)
    check(l, u, T=[1e-6, 1e-3, 50.0, 1e6], p=0.9)


def test_strided_rows_and_another_stream():
    l, u, r = rows(5, 4000, 15)
    wide = torch.from_numpy(l).cuda()
    check(wide[:, 3:3900], u, k=50, stream=torch.cuda.Stream())
    half = wide.to(torch.bfloat16)
    check(half[:, 1:1778], u, p=0.9)


def test_repeats_are_equal():
    from block_quantized_int8_gb300 import q8
    l, u, r = rows(33, 100003, 16)
    a = draw(l, u, T=0.8, k=200, p=0.9, m=0.01)
    for _ in range(5):
        b = draw(l, u, T=0.8, k=200, p=0.9, m=0.01)
        assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_frequencies_follow_the_distribution():
    # 20,000 draws of one row
    V, n = 12, 20000
    l = np.linspace(-2, 2, V, dtype=np.float32)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tok, _, _ = draw(np.tile(l, (n, 1)), u)
    p = np.exp(l.astype(np.float64))
    p /= p.sum()
    # u is an even grid: counts are within two of n p
    assert np.all(np.abs(np.bincount(tok, minlength=V) - n * p) <= 2)
