"""Float64 oracle of the linear layers in 8-bit floating point (test infrastructure).

Codes are bytes in e4m3 (sign, 4 exponent bits with bias 7, 3 of mantissa; 0x7F and 0xFF are
NaN, there are no infinities); rows have a scale for each 128 columns, [ceil(K/128), M],
weights one for each block of 128 x 128."""
import numpy as np

TINY = 2.0 ** -117


def decode(codes):
    b = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(8.0 + m, e - 10), np.ldexp(m.astype(np.float64), -9))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


def half_step(y):
    """Half the distance of e4m3 neighbours at |y| (2^-10 below the smallest normal number)."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return np.exp2(np.minimum(e, 8) - 4)


def encode(y):
    """Nearest e4m3 code, ties to even, saturating at 448."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 448.0)
    step = 2 * half_step(np.where(np.isfinite(a), a, 0.0))
    r = np.minimum(np.rint(np.where(np.isnan(a), 0.0, a) / step) * step, 448.0)
    e = np.floor(np.log2(np.maximum(r, 2.0 ** -6))).astype(np.int64)
    sub = r < 2.0 ** -6
    code = np.where(sub, r * 512, (e + 7) * 8 + np.rint(np.ldexp(r, 3 - e)) - 8).astype(np.int64)
    code = np.where(np.isnan(y), 127, code)
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def blocks(n):
    return -(-n // 128)


def spread(scale, n, axis):
    """Scales repeated for the n elements along ``axis`` that they belong to."""
    return np.take(np.repeat(scale, 128, axis=axis), np.arange(n), axis=axis)


def _maxima(a, axes):
    """Largest magnitude of each block of 128 along ``axes``."""
    for ax in axes:
        n = a.shape[ax]
        a = np.stack([np.take(a, np.arange(i, min(n, i + 128)), axis=ax).max(axis=ax)
                      for i in range(0, n, 128)], axis=ax)
    return a


def round_rows(h):
    """h [M, K]: (codes, scales [ceil(K/128), M])."""
    s = np.maximum(_maxima(np.abs(h), (1,)), TINY) / 448
    return encode(h / spread(s, h.shape[1], 1)), s.T.copy()


def round_weight(w):
    """w [.., N, K]: (codes, scales [.., ceil(N/128), ceil(K/128)])."""
    s = np.maximum(_maxima(np.abs(w), (w.ndim - 2, w.ndim - 1)), TINY) / 448
    return encode(w / spread(spread(s, w.shape[-2], w.ndim - 2), w.shape[-1], w.ndim - 1)), s


def rows_value(codes, scale):
    return decode(codes) * spread(np.asarray(scale, np.float64).T, codes.shape[1], 1)


def weight_value(codes, scale):
    s = np.asarray(scale, np.float64)
    return decode(codes) * spread(spread(s, codes.shape[-2], s.ndim - 2), codes.shape[-1],
                                  s.ndim - 1)


def norm_rows(x, residual=None, norm_w=None, eps=1e-6):
    """(s, h): the sum, and what is rounded to 8 bits."""
    s = x if residual is None else x + residual
    if norm_w is None:
        return s, s
    return s, s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * norm_w


def silu_mul(gate_up):
    g, u = np.split(gate_up, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def linear(x, w):
    """x [M, K], w [N, K] as values."""
    return x @ w.T


def grouped(x, w, start, rows, out):
    """``out`` with the rows of each expert written; of those that claim a row twice, the first's."""
    out = out.copy()
    m, end = len(out), 0
    for e in range(len(w)):
        a, b = int(start[e]), int(start[e + 1])
        if not 0 <= a <= b <= m or a < end and a < b:
            continue
        end = max(end, b) if a < b else end
        for n in range(a, b):
            src = n if rows is None else int(rows[n])
            out[n] = w[e] @ x[src] if 0 <= src < len(x) else 0.0
    return out
