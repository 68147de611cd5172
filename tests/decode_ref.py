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
