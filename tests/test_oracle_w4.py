"""Pins of the 4-bit oracle: published E2M1 values, brute-force nearest codes, error bounds, packing."""
import numpy as np
import pytest

from oracle import w4


def test_e2m1_values_are_the_formats():
    # sign | exponent (bias 1) | mantissa bit: 2^(e-1) (1 + m/2), subnormal m/2
    for c in range(8):
        e, m = c >> 1, c & 1
        assert w4.E2M1[c] == (m * 0.5 if e == 0 else 2.0 ** (e - 1) * (1 + m * 0.5))


@pytest.mark.parametrize("fmt,group", [("int4", 32), ("int4", 64), ("int4", 128), ("fp4", 32)])
def test_quantisation_error_and_extremes(fmt, group):
    r = np.random.default_rng(group)
    X = r.normal(size=(5, 256)) * np.exp(r.normal(size=(5, 256)))
    X[1] = 0.0
    X[2, :group] = 0.0
    codes, s = w4.quantize(X.astype(np.float32), fmt, group)
    V = w4.values(codes, s, fmt)
    assert np.all(V[1] == 0.0) and np.all(V[2, :group] == 0.0)
    g = np.abs(X.astype(np.float32).astype(np.float64)).reshape(5, -1, group)
    top = np.repeat(g.max(axis=2), group, axis=1)
    if fmt == "int4":  # half a step of s = top / 7 (1 + 2^-8), and what the clipping of 7 (1 + 2^-8) loses
        assert np.all(np.abs(V - X) <= top / 7 * (0.5 + 0.04) + 1e-12)
    else:  # top / s in (3, 6]: the widest gap is 2 s, half of it s < top / 3
        assert np.all(np.abs(V - X) <= top / 3 + 1e-12)
        e = np.repeat(2.0 ** (s.astype(np.float64) - 127), group, axis=1)
        assert np.all(top <= 6 * e) and np.all((top > 3 * e) | (top == 0))


def test_ties_go_to_the_even_code():
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [0.0] * 24])
    codes, s = w4.quantize(x, "fp4", 32)
    assert list(codes[0, :8]) == [7, 0, 2, 2, 4, 4, 6, 6] and s[0, 0] == 127
    x = np.array([[7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -7.0, 6.5] + [0.0] * 24])
    codes, s = w4.quantize(x, "int4", 32)
    assert s[0, 0] == 1.0 and list(codes[0, :8]) == [15, 8, 10, 10, 8, 6, 1, 14]


def test_packing_and_layout():
    c = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    assert w4.pack(c)[0, 0] == 0x10 and np.array_equal(w4.unpack(w4.pack(c)), c)
    s = np.arange(10).reshape(2, 5).astype(np.uint8)
    out = w4.store_scales(s, "fp4")
    assert out.shape == (2, 2, 4) and out[1, 1, 0] == 9 and out[1, 0, 1] == 127
    assert np.array_equal(w4.store_scales(s, "int4"), s.T)
