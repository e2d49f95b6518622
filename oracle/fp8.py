"""E4M3 codes with block scales, RMS norm, and the FP8 linear (oracle).

E4M3 is the OCP 8-bit format with 4 exponent bits (bias 7) and 3 mantissa
bits, no infinities, NaN at 0x7F / 0xFF, largest finite value 448 ([P5] names
FP8 deployment and its E4M3 layout; the scale granularities are readings):

  * activations: one fp32 scale per token and 128 consecutive values of k;
  * weights: one fp32 scale per block of 128 x 128;
  * s = max|v| / 448 (fp32 division), 1 for a block of zeros, at least the
    smallest normal fp32 value 2^-126;
  * code = E4M3(v / s): the fp32 division, then one rounding to nearest, ties
    to even.

Norm and gated product are defined in fp64.
"""

import numpy as np

from .numerics import f32

BLOCK = 128
MAX = np.float32(448.0)
TINY = np.float32(2.0 ** -126)


def decode_table():
    """fp64 values of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = c >> 7, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v = np.nan
        elif e == 0:
            v = m * 2.0 ** -9
        else:
            v = (8 + m) * 2.0 ** (e - 10)
        out[c] = -v if sign else v
    return out


_TABLE = decode_table()


def decode(codes):
    return _TABLE[np.asarray(codes, np.uint8)]


def encode(v32):
    """fp32 -> E4M3 codes, nearest, ties to the even code; finite |v| below 464."""
    v = np.asarray(v32, np.float64)
    a = np.abs(v)
    mags = _TABLE[:127]
    mid = (mags[:-1] + mags[1:]) / 2
    lo = np.searchsorted(mid, a, side="left")      # midpoints strictly below a
    hi = np.searchsorted(mid, a, side="right")     # ... or equal to it
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def scale_of(amax32):
    """The fp32 scale of a block whose largest magnitude is amax32."""
    a = np.asarray(amax32, np.float32)
    s = (a / MAX).astype(np.float32)
    return np.where(a == 0, np.float32(1), np.maximum(s, TINY)).astype(np.float32)


def _codes(v, s):
    return encode((v / s).astype(np.float32))


def quantize_rows(v32):
    """fp32 [m][k] -> (codes [m][k], scales fp32 [ceil(k/128)][m])."""
    v = f32(v32)
    m, k = v.shape
    kb = -(-k // BLOCK)
    codes = np.zeros((m, k), np.uint8)
    scales = np.zeros((kb, m), np.float32)
    for b in range(kb):
        cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
        scales[b] = scale_of(np.abs(v[:, cols]).max(axis=1))
        codes[:, cols] = _codes(v[:, cols], scales[b][:, None])
    return codes, scales


def quantize_block(w16):
    """16-bit weights [n][k] -> (codes [n][k], scales fp32 [ceil(n/128)][ceil(k/128)])."""
    w = f32(w16)
    n, k = w.shape
    codes = np.zeros((n, k), np.uint8)
    scales = np.zeros((-(-n // BLOCK), -(-k // BLOCK)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            scales[i, j] = scale_of(np.abs(w[at]).max())
            codes[at] = _codes(w[at], scales[i, j])
    return codes, scales


def dequantize_rows(codes, scales):
    k = codes.shape[1]
    return decode(codes) * np.repeat(np.asarray(scales, np.float64).T, BLOCK, axis=1)[:, :k]


def dequantize_block(codes, scales):
    n, k = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), BLOCK, 0)[:n], BLOCK, 1)[:, :k]
    return decode(codes) * s


def add_rmsnorm(x, gain, eps, residual=None):
    """fp64 (h, v) of given values."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rms = np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h, h / rms * np.asarray(gain, np.float64)


def silu_product(x, up):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x)) * np.asarray(up, np.float64)
