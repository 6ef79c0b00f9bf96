"""The operators between a decoder layer's linears, the plain way (test
infrastructure): RMS norm, E4M3 rows with one scale, rotary positions, attention
of one token.  numpy; float64, or float32 step by step where the library's
definition is in float32.

Parity: pinned by tests/test_oracle_layer.py (pure-Python loops, exact
rationals, complex rotation, torch's E4M3 cast, softmax identities).
"""

import numpy as np

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100


def e4m3_round(x):
    """Float64 values of the E4M3 codes nearest to x (ties to even, saturating)."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
        step = np.exp2(np.maximum(e.astype(np.float64) - 4, -9.0))
        return np.clip(np.rint(x / step) * step, -E4M3_MAX, E4M3_MAX)


def quantise(y):
    """(values of the codes, scales) of rows (last axis) of float32 y, in the
    float32 steps of the definition: s = max(amax / 448, 2^-100), E4M3(y / s).
    NaN entries do not enter amax."""
    y = np.asarray(y, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.fmax.reduce(np.abs(y), axis=-1, initial=np.float32(0))
        s = np.maximum(amax / np.float32(E4M3_MAX), np.float32(MIN_SCALE)).astype(np.float32)
        return e4m3_round((y / s[..., None]).astype(np.float32)), s


def rms_norm(x, weight, eps):
    """x * rsqrt(mean(x^2) + eps) * weight over the last axis, float64."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(all="ignore"):
        return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def axis_of_frequency(sections):
    return np.repeat(np.arange(len(sections)), sections)


def rope(x, positions, table, sections=None, interleaved=False):
    """x [T, heads, D] rotated, float32, every product and sum rounded on its own.
    positions [axes, T]; a position outside the table leaves its elements."""
    x = np.asarray(x, dtype=np.float32)
    out = x.copy()
    rot = table.shape[1]
    half = rot // 2
    axis = axis_of_frequency([half] if sections is None else sections)
    for f in range(half):
        p = positions[axis[f]]
        ok = (p >= 0) & (p < table.shape[0])
        q = np.where(ok, p, 0)
        c = np.where(ok, table[q, f], np.float32(1))[:, None]
        s = np.where(ok, table[q, half + f], np.float32(0))[:, None]
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        out[:, :, i] = x[:, :, i] * c - x[:, :, j] * s
        out[:, :, j] = x[:, :, j] * c + x[:, :, i] * s
    return out


def attend(q, k, v, scale):
    """One sequence: q [Hq, D], k and v [n, heads, D] -> out [Hq, D], lse [Hq] and
    sum_j p_j |v_j| (the magnitude that rounding errors of the weights scale with)."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    Hq, D = q.shape
    if k.shape[0] == 0:
        return np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros((Hq, D))
    G = Hq // k.shape[1]
    out, lse, mag = np.empty((Hq, D)), np.empty(Hq), np.empty((Hq, D))
    for h in range(Hq):
        z = scale * (k[:, h // G] @ q[h])
        m = z.max()
        w = np.exp(z - m)
        total = w.sum()
        out[h] = w @ v[:, h // G] / total
        mag[h] = w @ np.abs(v[:, h // G]) / total
        lse[h] = m + np.log(total)
    return out, lse, mag
