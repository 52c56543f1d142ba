"""Float64 oracles of the operators around the head: token embedding, residual RMS norm and
8-bit checkpoint rows, written from the definitions (numpy; test infrastructure only)."""

from __future__ import annotations

import numpy as np

Q_BLOCK = 128


def round_e4m3(x):
    """Nearest e4m3 value (ties to even) of float64 x with |x| <= 448; non-finite x gives NaN."""
    x = np.asarray(x, np.float64)
    out = np.full(x.shape, np.nan)
    f = np.isfinite(x)
    a = np.abs(x[f])
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    e = np.maximum(e, -6.0)                       # below 2^-6: subnormal, step 2^-9
    step = np.exp2(e - 3)
    out[f] = np.rint(x[f] / step) * step
    assert np.all(np.abs(out[f]) <= 448.0)
    return out


def block_exponent(x):
    """Per row and 128 columns: e of the smallest 2^e >= 2^-117 with |x| <= 448 * 2^e over the
    finite elements; 0 for a block of zeros. [N, ceil(H/128)]."""
    x = np.asarray(x, np.float64)
    N, H = x.shape
    nb = (H + Q_BLOCK - 1) // Q_BLOCK
    e = np.zeros((N, nb))
    for b in range(nb):
        a = np.abs(x[:, b * Q_BLOCK:(b + 1) * Q_BLOCK])
        m = np.where(np.isfinite(a), a, 0.0).max(axis=1)
        mant, ex = np.frexp(m)                    # m = mant * 2^ex, mant in [0.5, 1); 448 = 0.875 * 2^9
        e[:, b] = np.where(m > 0, np.maximum(ex - 9 + (mant > 0.875), -117), 0)
    return e


def spread(s, H):
    """Block values [N, nb] over H columns."""
    return np.repeat(s, Q_BLOCK, axis=1)[:, :H]


def pack(x):
    """(q, scale) of an array; q as the e4m3 values."""
    s = np.exp2(block_exponent(x))
    return round_e4m3(np.asarray(x, np.float64) / spread(s, x.shape[1])), s


def embed_fwd(tokens, E, scale, ignore_index):
    out = np.zeros((tokens.size, E.shape[1]))
    for i, t in enumerate(tokens):
        if t != ignore_index and 0 <= t < E.shape[0]:
            out[i] = scale * E[t]
    return out


def embed_bwd(tokens, dout, V, scale, ignore_index):
    """(dE, sum of magnitudes, rows per token)."""
    dE = np.zeros((V, dout.shape[1]))
    mag = np.zeros_like(dE)
    n = np.zeros(V, np.int64)
    for i, t in enumerate(tokens):
        if t != ignore_index and 0 <= t < V:
            dE[t] += scale * dout[i]
            mag[t] += np.abs(scale * dout[i])
            n[t] += 1
    return dE, mag, n


def rmsnorm_fwd(h, w, eps, off):
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * (w + off), rstd


def rmsnorm_bwd(dy, h, rstd, w, off, dh=None):
    """dx, dweight, and the magnitudes that enter their error bounds."""
    xh = h * rstd[:, None]
    g = dy * (w + off)
    m = np.mean(g * xh, axis=1, keepdims=True)
    dx = rstd[:, None] * (g - xh * m)
    mag = rstd[:, None] * (8 * np.abs(g) + 80 * np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    if dh is not None:
        dx = dx + dh
        mag = mag + 4 * np.abs(dh)
    return dx, (dy * xh).sum(axis=0), mag, np.abs(dy * xh).sum(axis=0)
