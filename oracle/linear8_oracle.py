"""The 8-bit projections in float64 on the CPU: test infrastructure only."""
from __future__ import annotations

import numpy as np

# the value of each e4m3 code (bias 7, subnormals m * 2^-9, 0x7f and 0xff NaN)
VALUES = np.array([np.nan if c & 127 == 127 else
                   (-1) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if not c & 0x78 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                   for c in range(256)])
GRID = VALUES[:127]


def encode(x):
    """Codes of the nearest e4m3 values, ties to the even code; |x| <= 448 or not finite (0x7f)."""
    a = np.abs(np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0))
    hi = np.minimum(np.searchsorted(GRID, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isfinite(x), code | np.where(np.signbit(x), 128, 0), 127).astype(np.uint8)


def scale_byte(amax):
    """Exponent byte of the least power of two s with amax <= 448 s, 2^-126 at least."""
    m, e = np.frexp(amax)
    e = np.where(m > 0.875, e - 8, e - 9)
    return np.where(amax > 0, np.maximum(e, -126) + 127, 1).astype(np.uint8)


def spread(s, high, R, K):
    """Scales of the elements of an [R, K] matrix, from exponent bytes (255: NaN)."""
    s = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return s.repeat(high, 0)[:R].repeat(128, 1)[:, :K]


def quantize(x, high=1):
    """(codes, exponent bytes) of x [R, K] in blocks of high x 128."""
    R, K = x.shape
    pad = np.zeros((-(-R // high) * high, -(-K // 128) * 128))
    pad[:R, :K] = np.where(np.isfinite(x), np.abs(x), 0)
    s = scale_byte(pad.reshape(pad.shape[0] // high, high, -1, 128).max((1, 3)))
    return encode(x / spread(s, high, R, K)), s


def values(codes, s, high=1):
    return VALUES[codes] * spread(s, high, *codes.shape)


def silu_mul(x):
    gate, up = np.split(x, 2, 1)
    with np.errstate(over="ignore"):
        return gate / (1 + np.exp(-gate)) * up


def rms_norm(h, w, eps):
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return y if w is None else y * w


def linear(a, w):
    """(A W^T, |A| |W|^T): the sums and the size of what is summed."""
    return a @ w.T, np.abs(a) @ np.abs(w).T
