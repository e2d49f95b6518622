"""Pins of the FP8, norm and mixture-of-experts oracles (CPU)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from exact_fp import FP32, exact, rn
from oracle import fp8, moe


def test_e4m3_values_and_codes():
    t = fp8.decode_table()
    assert t[0] == 0 and t[0x7E] == 448 and t[0x08] == 2.0 ** -6 and t[0x01] == 2.0 ** -9
    assert t[0x38] == 1.0 and t[0x39] == 1.125 and t[0xB8] == -1.0
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF])
    assert np.all(np.diff(t[:127]) > 0)
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref, equal_nan=True)
    fin = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(fp8.encode(t[fin].astype(np.float32)), fin)


def test_e4m3_rounding_is_nearest_even():
    r = np.random.default_rng(3)
    t = fp8.decode_table()[:127]
    mid = ((t[:-1] + t[1:]) / 2).astype(np.float32)       # exact in fp32
    near = np.concatenate([mid, np.nextafter(mid, np.float32(0)),
                           np.nextafter(mid, np.float32(1000)),
                           r.uniform(-448, 448, 4000).astype(np.float32),
                           (r.uniform(-1, 1, 4000) * 2.0 ** -6).astype(np.float32)])
    near = np.concatenate([near, -near])
    assert np.array_equal(fp8.encode(mid) % 2, np.zeros(126))
    ref = torch.from_numpy(near).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(near), ref)


def test_scales():
    assert fp8.scale_of(np.float32(0)) == 1
    assert fp8.scale_of(np.float32(448)) == 1
    assert fp8.scale_of(np.float32(1e-42)) == np.float32(2.0 ** -126)
    a = np.float32(0.7)
    exact = Fraction(float(a)) / 448
    assert abs(Fraction(float(fp8.scale_of(a))) - exact) <= exact / 2 ** 24


def test_row_and_block_layouts():
    r = np.random.default_rng(4)
    v = r.standard_normal((5, 300)).astype(np.float32)
    v[2, 128:256] = 0
    codes, s = fp8.quantize_rows(v)
    assert s.shape == (3, 5) and s[1, 2] == 1 and not codes[2, 128:256].any()
    err = np.abs(fp8.dequantize_rows(codes, s) - v)
    # half a step: a sixteenth of the value, or 2^-10 of the scale below 2^-6 of it
    assert np.all(err <= np.maximum(np.abs(v) / 16, s.T.repeat(128, 1)[:, :300] * 2.0 ** -10) * 1.0001)
    w = r.standard_normal((200, 144)).astype(np.float16)
    codes, s = fp8.quantize_block(w)
    assert s.shape == (2, 2)
    # a block's codes are those of the block alone
    c1, s1 = fp8.quantize_block(w[128:, 128:])
    assert s1[0, 0] == s[1, 1] and np.array_equal(c1, codes[128:, 128:])
    d = fp8.dequantize_block(codes, s)
    assert np.abs(d[130, 5] - float(w[130, 5])) <= max(abs(float(w[130, 5])) / 16, s[1, 0] / 1024) * 1.0001


def test_norm():
    h, v = fp8.add_rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0)
    rms = math.sqrt(12.5)
    assert np.allclose(v, [[3 / rms, 8 / rms]], rtol=1e-15)
    h, v = fp8.add_rmsnorm([[1.0, 1.0]], [1.0, 1.0], 0.0, [[2.0, 3.0]])
    assert np.array_equal(h, [[3.0, 4.0]]) and np.allclose(v, [[3 / rms, 4 / rms]], rtol=1e-15)
    # scale invariance without eps
    x = np.random.default_rng(5).standard_normal((2, 64))
    assert np.allclose(fp8.add_rmsnorm(x, np.ones(64), 0.0)[1],
                       fp8.add_rmsnorm(8 * x, np.ones(64), 0.0)[1], rtol=1e-13)


def test_silu_product():
    assert np.allclose(fp8.silu_product([math.log(3)], [4.0]), [3 * math.log(3)])
    assert fp8.silu_product([-2000.0], [1.0])[0] == 0


def test_routing():
    inf = np.inf
    ids, p = moe.route([[0.0, 1.0, 1.0, -inf]], 3, False)
    assert ids.tolist() == [[1, 2, 0]]
    e = math.e
    assert np.allclose(p, [[e / (1 + 2 * e), e / (1 + 2 * e), 1 / (1 + 2 * e)]])
    _, p = moe.route([[0.0, 1.0, 1.0, -inf]], 2, True)
    assert np.allclose(p, 0.5)
    ids, p = moe.route([[-inf, -inf, 2.0]], 2, True)
    assert ids.tolist() == [[2, 0]] and p.tolist() == [[1.0, 0.0]]
    ids, p = moe.route([[-inf, -inf]], 1, True)
    assert ids.tolist() == [[0]] and p.tolist() == [[0.0]]


@pytest.mark.parametrize("renorm", [True, False])
def test_experts_against_loops(renorm):
    r = np.random.default_rng(6)
    t, e, h, i = 3, 4, 5, 6
    x = r.standard_normal((t, h))
    g, u, d = (r.standard_normal(s) for s in ((e, i, h), (e, i, h), (e, h, i)))
    ids, p = moe.route(r.standard_normal((t, e)), 2, renorm)
    y = moe.experts(x, ids, p, g, u, d)
    for a in range(t):
        for o in range(h):
            s = 0.0
            for j in range(2):
                ex = ids[a, j]
                for c in range(i):
                    gv = sum(g[ex, c, q] * x[a, q] for q in range(h))
                    uv = sum(u[ex, c, q] * x[a, q] for q in range(h))
                    s += p[a, j] * d[ex, o, c] * gv / (1 + math.exp(-gv)) * uv
            assert abs(s - y[a, o]) <= 1e-12 * (1 + abs(s))


def row_of(v):
    """[v] as the rows of a block 128 wide, zeros behind."""
    out = np.zeros((1, 128), np.float32)
    out[0, :len(v)] = v
    return out


# The code is that of the fp32 quotient v / s; v times the reciprocal of s gives
# the neighbouring one here.
@pytest.mark.parametrize("amax,v,code", [(1.078125, 0.80859375, 122), (1.0234375, 0.767578125, 122),
                                         (1.03125, 1.5735626220703125e-05, 4)])
def test_codes_are_of_the_quotient(amax, v, code):
    a, x = np.float32(amax), np.float32(v)
    s = np.float32(a / np.float32(448))
    near = np.float32(float(rn(exact(x) / exact(s), FP32)))
    assert fp8.encode(near) == code
    assert fp8.encode(np.float32(x * (np.float32(1) / s))) != code
    codes, _ = fp8.quantize_rows(row_of([a, x, -x]))
    assert codes[0, :3].tolist() == [126, code, code | 128]
    codes, _ = fp8.quantize_block(row_of([a, x, -x]).astype(np.float16).repeat(2, 0))
    assert codes[1, :3].tolist() == [126, code, code | 128]


def fma(a, b, c):
    """fp32 fused multiply-add of scalars, rounded once."""
    v = exact(a) * exact(b) + exact(c)
    if v == 0:
        return np.float32(float(a) * float(b) + float(c))    # the sign of zero
    return np.float32(float(rn(v, FP32)))


def corrected(v, s, inv):
    """v / s as the packers divide in fp32: v * inv and its residual times inv."""
    q = v * inv
    return fma(-fma(q, s, -v), inv, q)


def reciprocals(s):
    """1 / s from a reciprocal up to one step off, with its residual added."""
    near = np.float32(1) / s
    for start in (near, np.nextafter(near, np.float32(0)), np.nextafter(near, 2 * near)):
        yield fma(fma(-s, start, np.float32(1)), start, start)


def test_a_corrected_quotient_has_the_codes_of_the_division():
    """v * inv is off by at most 2.5 steps even if inv is off by one; with its
    residual times inv, 2^-21 of a step is left.  That can change an fp32 rounding
    only next to a midpoint of two fp32 values, and a code only where that midpoint
    is half a step from a midpoint of two codes (5 bits).  With integers A / B of 24
    bits that takes B within 13 of a multiple of 2^20: those scales, each with the
    values around every midpoint."""
    n = 0
    for c in range(8, 17):
        for delta in range(-14, 15):
            B = (c << 20) + delta
            if B < 1 << 23 or B >= 1 << 24:
                continue
            s = np.float32(B)
            for j in range(17, 32, 2):
                for A in range(B * j // 32 - 2, B * j // 32 + 4):
                    v = np.float32(A)
                    code = fp8.encode(np.float32(v / s))
                    for inv in reciprocals(s):
                        assert fp8.encode(corrected(v, s, inv)) == code, (A, B)
                        n += 1
    assert n > 30000
    r = np.random.default_rng(8)
    v = np.float32(r.uniform(1, 2, 1000))
    s = np.float32(r.uniform(1, 2, 1000) * 2.0 ** -4)
    for a, b in zip(v, s):
        for inv in reciprocals(b):
            assert fp8.encode(corrected(a, b, inv)) == fp8.encode(a / b)
    for zero in (np.float32(0.0), np.float32(-0.0)):
        for inv in reciprocals(np.float32(3)):
            assert np.signbit(corrected(zero, np.float32(3), inv)) == np.signbit(zero)


def test_a_corrected_scale_is_the_division():
    """a * (1 / 448) and its residual, for every mantissa; fp64 holds each step but
    the last sum, which is rounded far from a midpoint."""
    inv = np.float32(1) / np.float32(448)
    for part in np.split(np.arange(1 << 23, 1 << 24), 8):
        a = part.astype(np.float32)
        q = a * inv
        r = (a.astype(np.float64) - q.astype(np.float64) * 448).astype(np.float32)
        got = (r.astype(np.float64) * np.float64(inv) + q).astype(np.float32)
        assert np.array_equal(got, a / np.float32(448))
