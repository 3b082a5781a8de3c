"""Oracle of decode over selected key blocks: bounds of blocks of 64 keys, the
choice of a query's blocks by a score of those bounds, and attention over the
listed blocks.

TEST INFRASTRUCTURE ONLY (same rules as the rest of `oracle/`): it shares no
code with the CUDA library and never imports it.

Bounds of a block with keys x [64, 256], in float32: hi / lo = the largest /
smallest value of each dim (NaN where one of them is), scale = max(|hi|, |lo|)
* f32(1/127), codes = clamp(round_half_even(x / scale), -127, 127) of hi and lo
(0 where the scale is not finite or not positive) -- the rule of `quant`.

Score of block j for the 8 query rows (codes q8, scales sq):

    s_j = max_h f32(sum_t (q8_t > 0 ? q8_t hi8_t : q8_t lo8_t)) * (sq_h * scale_j)

in float32, NaN above all numbers.  The first n_sink and last n_recent of the
ceil(ctx / 64) blocks are taken, then the highest scores, ties by lower index.
The pages have no such calls.
"""
import numpy as np

from .partial import widen
from .quant import INV127, quantize_rows, widen32

KEYS = 64


def bounds(x32):
    """x32 [64, 256] float32 -> codes int8 [2, 256], scale float32."""
    with np.errstate(invalid="ignore"):
        both = np.stack((x32.max(0), x32.min(0))).astype(np.float32)   # numpy's max and min keep NaN
    codes, scale = quantize_rows(both.reshape(1, 512))
    return codes.reshape(2, 256), scale.reshape(())


def summarize(k, kv_dtype, ctx, n_new, codes, scales):
    """Copies of codes / scales with the blocks that the newest n_new positions
    of each sequence finished; a length outside 0..capacity changes nothing."""
    codes, scales = codes.copy(), scales.copy()
    x = widen32(k, kv_dtype)
    for b, c in enumerate(ctx):
        if c < 0 or c > x.shape[1]:
            continue
        for j in range(scales.shape[1]):
            if c - n_new < KEYS * (j + 1) <= c:
                codes[b, j], scales[b, j] = bounds(x[b, KEYS * j:KEYS * (j + 1)])
    return codes, scales


def scores(q, q_dtype, codes, scales, n):
    """float32 scores [n] of the first n blocks; q [8, 256], codes [>= n, 2, 256]."""
    q8, sq = quantize_rows(widen32(q, q_dtype))
    q8 = q8.astype(np.int64)
    hi, lo = codes[:n, 0].astype(np.int64), codes[:n, 1].astype(np.int64)
    dot = np.maximum(q8, 0) @ hi.T + np.minimum(q8, 0) @ lo.T          # [8, n], exact
    with np.errstate(invalid="ignore", over="ignore"):
        s = dot.astype(np.float32) * (sq.reshape(8, 1).astype(np.float32) * scales[None, :n].astype(np.float32))
    return s.max(0)


def select(q, q_dtype, codes, scales, ctx, n_select, n_sink=1, n_recent=1):
    """The list of one sequence: ascending block indices, then -1."""
    n = -(-ctx // KEYS)
    forced = [j for j in range(n) if j < n_sink or j >= n - n_recent]
    if n <= n_select:
        ids = list(range(n))
    else:
        s = scores(q, q_dtype, codes, scales, n - 1)
        key = [(0 if np.isnan(s[j]) else 1, 0.0 if np.isnan(s[j]) else -float(s[j]), j)
               for j in range(n - 1) if j not in forced]
        ids = sorted(forced + [j for _, _, j in sorted(key)[:n_select - len(forced)]])
    return ids + [-1] * (n_select - len(ids))


def attend(q, q_dtype, k, v, kv_dtype, blocks, ctx, scale=1.0 / 16.0):
    """One sequence: q [8, 256], k / v [capacity, 256], blocks: a list of block
    indices (-1 and blocks past the context hold no key).  Returns out float64
    [8, 256], the largest scale * sum |q||k| over the keys per head [8] and the
    largest |v| among the seen keys."""
    qd, kd, vd = widen(q, q_dtype), widen(k, kv_dtype), widen(v, kv_dtype)
    rows = [p for j in blocks if j >= 0 for p in range(KEYS * j, min(ctx, KEYS * (j + 1)))]
    out = np.zeros((8, 256))
    if not rows:
        return out, np.zeros(8), 0.0
    s = scale * (qd @ kd[rows].T)
    w = np.exp(s - s.max(1, keepdims=True))
    out = (w @ vd[rows]) / w.sum(1, keepdims=True)
    return out, scale * (np.abs(qd) @ np.abs(kd[rows]).T).max(1), float(np.abs(vd[rows]).max())
