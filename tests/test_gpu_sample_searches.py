"""q8_sample where a list of few words will not do: the searches of top-k and top-p over the
whole row, at temperatures on both sides of one.  The check is test_gpu_sample's."""
import numpy as np
import pytest

import test_gpu_sample as sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0.01, 0.3, 2.0, 4.0, 50.0, 1e20])
@pytest.mark.parametrize("V,k", [(4096, 2000), (32003, 1500), (32003, 30000), (131071, 5000)])
def test_top_k_over_the_whole_row(T, V, k):
    # logits spread over about 60 T, evenly or with a peak far above the others
    r = np.random.default_rng(V + k)
    l = np.empty((4, V), dtype=np.float32)
    l[0] = np.linspace(0.0, -60.0 * T, V)
    l[1] = r.permutation(l[0])
    l[2:] = r.standard_normal((2, V)) * 4.0 * T
    l[2:, V // 3] = 30.0 * T
    sample.check(l, r.random(4).astype(np.float32), T=T, k=k, p=[1.0, 0.9, 1.0, 0.999999])


def test_top_k_with_one_word_far_above_the_others():
    r = np.random.default_rng(1)
    l = (r.standard_normal((8, 32000)) * 3.0).astype(np.float32)
    l[:, 7000] = 35.0
    tok, lp, kept = sample.check(l, r.random(8).astype(np.float32), T=[2.0, 2.0, 4.0, 4.0, 10.0, 2.5, 3.0, 8.0], k=2000)
    assert kept.tolist() == [2000] * 8


@pytest.mark.parametrize("T", [0.5, 2.0, 20.0])
@pytest.mark.parametrize("k", [3, 40, 500, 1000])
def test_top_k_among_many_equal_words(T, k):
    # more equal words at the last place than a list holds; the peak lies 40 T above them
    r = np.random.default_rng(k)
    l = np.full((3, 20000), -40.0 * T, dtype=np.float32)
    l[:, ::2] = -80.0 * T
    l[1, r.permutation(20000)[:2]] = 0.0
    l[2] += r.integers(0, 2, 20000).astype(np.float32) * T
    sample.check(l, r.random(3).astype(np.float32), T=T, k=k, p=[1.0, 1.0, 0.7])


@pytest.mark.parametrize("V", [1, 2, 64, 65, 500, 1000, 1001, 3000])
@pytest.mark.parametrize("p", [1.0, 1.0 + 2.0 ** -23, 1.5, 1e30, np.inf, np.nan])
def test_top_p_of_one_and_more_keeps_all_words(V, p):
    # the same draw as without top-p, whether or not the vocabulary fits a list; logits of both signs
    l, u, r = sample.rows(6, V, V)
    l[1] += 20.0
    l[2] -= 20.0
    l[3, : V // 2] = -np.inf
    for k in (0, V, 40):
        a = sample.draw(l, u, T=[1.0, 0.7, 1.3, 1.0, 0.0, 2.0], k=k, p=p)
        b = sample.check(l, u, T=[1.0, 0.7, 1.3, 1.0, 0.0, 2.0], k=k)
        assert all(np.array_equal(x, y) for x, y in zip(a, b)), (k, a, b)


@pytest.mark.parametrize("V", [2049, 5000, 32003, 131071])
def test_top_k_around_the_places_where_the_search_changes(V):
    # by the k-th group maximum up to 96, by a rank among them up to 1152, by the histogram above
    r = np.random.default_rng(V)
    k = np.array([1, 63, 64, 65, 95, 96, 97, 127, 128, 129, 170, 171, 999, 1000, 1001, 1151, 1152, 1153, 1366, 2047])
    l = (r.standard_normal((len(k), V)) * 2.5).astype(np.float32)
    for p in (1.0, 0.9):
        tok, lp, kept = sample.check(l, r.random(len(k)).astype(np.float32), T=0.8, k=k, p=p)
        assert p < 1.0 or np.array_equal(kept, k)
