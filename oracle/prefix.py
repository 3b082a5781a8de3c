"""Oracle of decode over a prefix that a batch shares: sequence b sees the
positions [max(0, ctx - window), ctx) (all before ctx without a window), those
below prefix_len in the one prefix, the others in its own cache.

TEST INFRASTRUCTURE ONLY (same rules as the rest of `oracle/`): it shares no
code with the CUDA library and never imports it.  The pages have no such call;
the arithmetic is plain softmax attention in float64, an empty row exactly 0.
"""
import numpy as np

from .partial import widen


def attend(q, q_dtype, pk, pv, k, v, kv_dtype, ctx, window=0, scale=1.0 / 16.0):
    """One sequence: q [8, 256], pk / pv [prefix_len, 256], k / v [capacity, 256].
    Returns out [8, 256], the largest scale * sum |q||k| per head [8], the largest
    |v| seen, sum p |v| / sum p [8, 256] and the number of keys."""
    lo = max(0, ctx - window) if window > 0 else 0
    n = pk.shape[0]
    kk = np.concatenate((widen(pk[lo:], kv_dtype), widen(k[max(0, lo - n):max(0, ctx - n)], kv_dtype)))
    vv = np.concatenate((widen(pv[lo:], kv_dtype), widen(v[max(0, lo - n):max(0, ctx - n)], kv_dtype)))
    if kk.shape[0] == 0:
        return np.zeros((8, 256)), np.zeros(8), 0.0, np.zeros((8, 256)), 0
    qd = widen(q, q_dtype)
    s = scale * (qd @ kk.T)
    p = np.exp(s - s.max(1, keepdims=True))
    l = p.sum(1, keepdims=True)
    return (p @ vv) / l, scale * (np.abs(qd) @ np.abs(kk).T).max(1), float(np.abs(vv).max()), (p @ np.abs(vv)) / l, len(kk)
