"""fp64 CPU oracle of the operators around and inside the block: the norms with
their gate and residual scales (forward and backward), rounding to e4m3 with a
scale for each block of 128, and the products of such rows and weights.

Plain NumPy, written from the formulas; nothing here is shared with the CUDA
library.
"""
import numpy as np

QMAX, SMIN = 448.0, 2.0 ** -126


# ------------------------------------------------------------------ norms

def norm_stats(x, kind, eps):
    """(mean, rstd) of each row, float64 [T, 1]; mean 0 for RMS; (0, 1) without a norm."""
    x = np.asarray(x, np.float64)
    zero = np.zeros((x.shape[0], 1))
    if kind == "none":
        return zero, zero + 1.0
    mean = x.mean(axis=1, keepdims=True) if kind == "layer" else zero
    return mean, 1.0 / np.sqrt(np.mean((x - mean) ** 2, axis=1, keepdims=True) + eps)


def norm(x, kind, eps, w=None, b=None, offset=0.0):
    x = np.asarray(x, np.float64)
    mean, rstd = norm_stats(x, kind, eps)
    y = (x - mean) * rstd
    if w is not None:
        y = y * (np.asarray(w, np.float64) + offset)
    return y if b is None else y + b


def norm_backward(x, dy, kind, eps, w=None, offset=0.0):
    """(dx, dw, db) of norm for an upstream dy."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    mean, rstd = norm_stats(x, kind, eps)
    xhat = (x - mean) * rstd
    g = dy if w is None else dy * (np.asarray(w, np.float64) + offset)
    if kind == "none":
        return g, None, None
    dx = g - xhat * np.mean(g * xhat, axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - np.mean(g, axis=1, keepdims=True)
    return rstd * dx, np.sum(dy * xhat, axis=0), np.sum(dy, axis=0)


def norm_residual(r, y, kind, eps, w=None, b=None, offset=0.0, gate=None, alpha=1.0, beta=1.0):
    """alpha r + beta gate N(y); gate: anything that broadcasts against [T, d]."""
    n = norm(y, kind, eps, w, b, offset)
    return alpha * np.asarray(r, np.float64) + beta * (1.0 if gate is None else gate) * n


def norm_residual_backward(y, dout, kind, eps, w=None, b=None, offset=0.0, gate=None, alpha=1.0, beta=1.0):
    """(dr, dy, dw, db, dgate at every element) for an upstream dout."""
    dout = np.asarray(dout, np.float64)
    n = norm(y, kind, eps, w, b, offset)
    d = beta * (1.0 if gate is None else gate) * dout
    dy, dw, db = norm_backward(y, d, kind, eps, w, offset)
    return alpha * dout, dy, dw, db, beta * dout * n


# ------------------------------------------------------------------ e4m3

def round_e4m3(v):
    """The nearest e4m3 value, ties to the even one, beyond 448 saturated; NaN stays NaN."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), QMAX)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3.0)
    return np.copysign(np.rint(a / step) * step, v)


def e4m3_values(bits):
    """Values of e4m3 bytes (sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7F and 0xFF: NaN)."""
    u = np.asarray(bits, np.uint8).astype(np.int64)
    e, f = (u >> 3) & 15, u & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(u & 128, -v, v)


def block_scale(amax):
    """fp32 scale of a block: amax / 448 in fp32, at least 2^-126."""
    s = np.asarray(amax, np.float32) / np.float32(QMAX)
    return np.where(s < np.float32(SMIN), np.float32(SMIN), s).astype(np.float32)


def quantize_rows(x):
    """(q values in units of the scale, scales [KB, R]) of fp32 rows, by the library's fp32 definition."""
    x = np.asarray(x, np.float32)
    R, K = x.shape
    q, s = np.empty((R, K)), np.empty(((K + 127) // 128, R), np.float32)
    for j in range(s.shape[0]):
        blk = x[:, 128 * j:128 * j + 128]
        s[j] = block_scale(np.abs(blk).max(axis=1))
        q[:, 128 * j:128 * j + 128] = round_e4m3((blk / s[j][:, None]).astype(np.float32))
    return q, s


def quantize_weights(w):
    """(q [N, K], scales [NB, KB]) of fp32 weights [N, K]."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    q, s = np.empty((N, K)), np.empty(((N + 127) // 128, (K + 127) // 128), np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = np.s_[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            s[i, j] = block_scale(np.abs(w[at]).max())
            q[at] = round_e4m3((w[at] / s[i, j]).astype(np.float32))
    return q, s


def dequantize_rows(q, s):
    K = q.shape[1]
    return np.asarray(q, np.float64) * np.repeat(np.asarray(s, np.float64), 128, axis=0)[:K].T


def dequantize_weights(q, s):
    N, K = q.shape
    return np.asarray(q, np.float64) * np.repeat(np.repeat(np.asarray(s, np.float64), 128, 0)[:N], 128, 1)[:, :K]


# ------------------------------------------------------------------ products

def matmul(a, offsets, weight):
    """Rows a [R, K] (values) times their expert's weight(e) [N, K]; rows past the last expert's: NaN."""
    a = np.asarray(a, np.float64)
    out = None
    for e in range(len(offsets) - 1):
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if out is None or r0 < r1:
            w = weight(e)
            if out is None:
                out = np.full((a.shape[0], w.shape[0]), np.nan)
            out[r0:r1] = a[r0:r1] @ w.T
    return out


def gated(g, u, limit):
    if limit > 0:
        g, u = np.clip(g, -limit, limit), np.clip(u, -limit, limit)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
