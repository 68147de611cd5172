"""Plain binary64 definitions of the decode-step operators, for the tests
(numpy; they share no code with the library)."""
import numpy as np


def values(q: np.ndarray, s_bits: np.ndarray) -> np.ndarray:
    """s * q of Q8_0 rows: codes int8 [..., K], binary16 scale bits [..., K / 32]."""
    s = s_bits.view(np.float16).astype(np.float64)
    return q.astype(np.float64) * np.repeat(s, 32, axis=-1)


def attention(q, k, v, scale, softcap=0.0, window=0):
    """One query row q[D] over keys k[n, D] and values v[n, D].  Returns (out[D], lse,
    sum_t p_t |v_t|, the largest sum_d |q_d k_d| * scale)."""
    n = k.shape[0]
    first = max(0, n - window) if window else 0
    k, v = k[first:], v[first:]
    if k.shape[0] == 0:
        return np.zeros(q.shape[0]), -np.inf, np.zeros(q.shape[0]), 0.0
    s = (k @ q) * scale
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    m = s.max()
    e = np.exp(s - m)
    p = e / e.sum()
    return p @ v, m + np.log(e.sum()), p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * abs(scale))


def route(logits, top_k, renorm):
    """One token's experts: (ids [top_k] with -1 for none, weights [top_k])."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    order = np.argsort(-l, kind="stable")[:top_k]
    ids = np.where(l[order] > -np.inf, order, -1)
    if ids[0] < 0:
        return ids, np.zeros(top_k)
    with np.errstate(invalid="ignore"):
        e = np.where(l == l.max(), 1.0, np.exp(l - l.max()))
    w = np.where(ids >= 0, e[order], 0.0)
    return ids, w / (w.sum() if renorm else e.sum())


def moe(x, logits, w13, w2, top_k, renorm):
    """Returns (y[T, H], bound[T, H], ids, weights).  The bound is what fp32 sums of K / 32
    blocks may be off (each block's product exact up to its own 32-term sum), carried
    through SwiGLU (silu's slope is below 1.1) and the down product, with 2^-20 of each
    hidden unit (exponential, division, product) and 2^-22 of its block's largest (how it is kept)."""
    T, H = x.shape
    F = w2.shape[2]
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    ids, ws = np.zeros((T, top_k), dtype=int), np.zeros((T, top_k))
    c1, c2 = (H / 32 + 40) * 2.0 ** -24, (F / 32 + 40) * 2.0 ** -24
    for t in range(T):
        ids[t], ws[t] = route(logits[t], top_k, renorm)
        for e, w in zip(ids[t], ws[t]):
            if e < 0:
                continue
            z, b = w13[e] @ x[t], np.abs(w13[e]) @ np.abs(x[t])
            a, u = z[:F], z[F:]
            with np.errstate(over="ignore"):
                s = a / (1 + np.exp(-a))
            act = s * u
            top = np.repeat(np.abs(act).reshape(-1, 32).max(1), 32)
            da = 1.1 * c1 * b[:F] * np.abs(u) + np.abs(s) * c1 * b[F:] + 2.0 ** -20 * np.abs(act) + 2.0 ** -22 * top
            y[t] += w * (w2[e] @ act)
            tol[t] += w * (np.abs(w2[e]) @ (da + c2 * np.abs(act)) + 2.0 ** -20 * np.abs(w2[e] @ act))
    return y, tol, ids, ws


def sample(logits, T, k, p, min_p, u):
    """One row, in binary64.  Returns (kept range, probability by word, total slack): the
    words kept are certain up to places where binary32 exponentials (2^-21 relative) could
    decide otherwise; the slack is the probability that hangs on those."""
    eps = 2.0 ** -20
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    V = l.shape[0]
    if not T > 0:
        T, k = 1.0, 1
    if k <= 0 or k > V:
        k = V
    m = l.max()
    if m == -np.inf:
        return (0, 0), np.zeros(V), 0.0
    with np.errstate(invalid="ignore"):
        e = np.where(l == m, 1.0, np.exp(np.where(l == m, 0.0, (l - m) / T)))
    e[l == -np.inf] = 0.0
    e = np.where(e >= 2.0 ** -40, e, 0.0)
    order = np.argsort(-l, kind="stable")
    r = e[order]
    r[k:] = 0.0
    total = r.sum()
    before = np.cumsum(r) - r
    sure = r > 2.0 ** -40 * (1 + eps)
    may = r > 0
    if p < 1.0:
        cut = max(p * total, 2.0 ** -40)
        sure &= before < cut - eps * total
        may &= before < cut + eps * total
        sure[0] = may[0]
    sure &= r >= min_p * (1 + eps)
    may &= r >= min_p * (1 - eps)
    if min_p <= 1.0:
        sure[0] = may[0] = r[0] > 0   # the largest has e = 1 exactly
    prob = np.zeros(V)
    both = np.where(may, r, 0.0)
    if both.sum() > 0:
        prob[order] = both / both.sum()
    slack = eps + (np.where(may & ~sure, r, 0.0).sum() / both.sum() if both.sum() > 0 else 0.0)
    return (int(sure.sum()), int(may.sum())), prob, slack
