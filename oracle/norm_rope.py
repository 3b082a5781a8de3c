"""Oracle of the fused norm + rotation + append: RMS norm of each head of q, of
k and of v, rotation by positions on several axes, q out, K / V into the cache.

TEST INFRASTRUCTURE ONLY (same rules as the rest of `oracle/`): it shares no
code with the CUDA library and never imports it.

For a row x of 256 values, in float64 from the exact stored values:

    y    = x / sqrt(mean(x^2) + eps) * (w + w0)
    a_i  = pos[axis_i] * inv_freq[i]                                 (i < 128)
    z_i  = y_i cos a_i - y_{i+128} sin a_i,  z_{i+128} = y_{i+128} cos a_i + y_i sin a_i

The pages have no such call (they hand cos/sin rows made on the host to the
append); the pairing of dim i with dim i + 128 is the append's.
"""
import numpy as np

from .partial import widen

HALF = 128


def norm(x, weight=None, w0=0.0, eps=1e-6):
    """RMS norm over the last axis; no weight and no offset when weight is None."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return y if weight is None else y * (weight + w0)


def turn(y, pos, inv_freq, axis):
    """Rotation of rows y [n, heads, 256] by pos [axes, n]; also returns the
    lengths of the pairs (what rounding errors of z are relative to)."""
    a = np.stack([pos[axis[i]].astype(np.float64) * float(inv_freq[i]) for i in range(HALF)], axis=-1)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    lo, hi = y[..., :HALF], y[..., HALF:]
    z = np.concatenate((lo * c - hi * s, hi * c + lo * s), axis=-1)
    r = np.hypot(lo, hi)
    return z, np.concatenate((r, r), axis=-1)


def norm_rope(q, k, v, dtype, *, pos=None, inv_freq=None, axis=None, wq=None, wk=None, w0=0.0, eps=1e-6,
              norm_qk=True, norm_v=False):
    """q [n, 8, 256], k / v [n, 256] in stored form, wq / wk float64 [256] or
    None, pos int64 [axes, n].  Returns (values, lengths): float64 [n, 10, 256]
    of the 8 query rows, the key and the value, and the pair lengths."""
    x = np.concatenate((widen(q, dtype), widen(k, dtype)[:, None], widen(v, dtype)[:, None]), axis=1)
    y = x.copy()
    if norm_qk:
        y[:, :8] = norm(x[:, :8], wq, w0, eps)
        y[:, 8] = norm(x[:, 8], wk, w0, eps)
    if norm_v:
        y[:, 9] = norm(x[:, 9], None, 0.0, eps)
    r = np.abs(y)
    if pos is not None:
        axis = [0] * HALF if axis is None else axis
        y[:, :9], r[:, :9] = turn(y[:, :9].copy(), np.asarray(pos), np.asarray(inv_freq), axis)
    return y, r
