"""The oracle of the gated block, the INT8 operands and gradient clipping against
facts from outside it: closed forms, differences, exact fractions."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import (act_ref, clip_ref, gated_backward_ref, gated_ref, int8_gemm_ref, int8_quantize_ref)


def test_activations_at_known_points():
    for act in ("silu", "gelu"):
        v, d = act_ref(np.array([0.0, 50.0, -50.0]), act)
        assert v[0] == 0 and d[0] == 0.5
        assert v[1] == 50.0 and abs(d[1] - 1) < 1e-15
        assert abs(v[2]) < 1e-18 and abs(d[2]) < 1e-18
    g = np.linspace(-6, 6, 101)
    assert np.allclose(act_ref(g, "silu")[0], g / (1 + np.exp(-g)), rtol=1e-14)
    # the tanh form is within 5e-4 of g Phi(g)
    exact = g * 0.5 * (1 + np.array([math.erf(x / math.sqrt(2)) for x in g]))
    assert np.abs(act_ref(g, "gelu")[0] - exact).max() < 5e-4


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes_against_differences(act):
    g = np.linspace(-9, 9, 361)
    step = 1e-5
    diff = (act_ref(g + step, act)[0] - act_ref(g - step, act)[0]) / (2 * step)
    assert np.abs(act_ref(g, act)[1] - diff).max() < 1e-9
    assert np.abs(act_ref(np.linspace(-20, 20, 400001), act)[1]).max() < 1.13


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward_against_differences(act):
    rng = np.random.default_rng(0)
    gu, dh = rng.standard_normal((3, 16)) * 2, rng.standard_normal((3, 8))

    def loss(x):
        return (act_ref(x[:, :8], act)[0] * x[:, 8:] * dh).sum()
    got, err = gated_backward_ref(dh, gu, act)
    for i in range(3):
        for j in range(16):
            up, dn = gu.copy(), gu.copy()
            up[i, j] += 1e-6
            dn[i, j] -= 1e-6
            assert abs((loss(up) - loss(dn)) / 2e-6 - got[i, j]) < 1e-7
    assert (err >= 0).all() and (err < 1e-4).all()


def test_gated_of_one_hot_operands():
    """x picks one column of W: g and u are single weights."""
    K, F = 32, 4
    x = np.zeros((K, K), np.uint8)
    x[np.arange(K), np.arange(K)] = 0x38                       # 1.0
    w = np.random.default_rng(1).integers(0, 0x7F, (2 * F, K)).astype(np.uint8)
    one = np.ones((1, K), np.float32)
    h, g, u, _, _ = gated_ref(x, one, w, np.ones((1, 2 * F), np.float32), 1, "silu")
    from oracle import E4M3_TABLE
    v = E4M3_TABLE[w]
    assert np.array_equal(g, v[:F].T) and np.array_equal(u, v[F:].T)
    assert np.allclose(h, v[:F].T / (1 + np.exp(-v[:F].T)) * v[F:].T, rtol=1e-14)


def test_int8_quantize_by_fractions():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((20, 48)) * np.exp2(rng.integers(-30, 30, (20, 1)))).astype(np.float32)
    x[3] = 0
    x[4, :] = np.float32(1.0) / np.float32(3.0)
    q, s = int8_quantize_ref(x)
    assert (np.abs(q.astype(int)).max(axis=1)[[i for i in range(20) if i != 3]] == 127).all()
    assert (q[3] == 0).all() and s[3] == np.float32(2.0 ** -100) / np.float32(127)
    for i in range(20):
        A = max(Fraction(float(np.abs(x[i]).max())), Fraction(1, 2 ** 100))
        assert s[i] == np.float32(float(A) / 127)
        r = Fraction(float(np.float32(127.0 / float(A))))
        for k in range(48):
            v = np.float32(float(Fraction(float(x[i, k])) * r))
            want = round(Fraction(float(v)))                 # to even at ties
            assert q[i, k] == want
    bad = x.copy()
    bad[1, 5], bad[2, 0] = np.nan, -np.inf
    q, s = int8_quantize_ref(bad)
    assert np.isnan(s[[1, 2]]).all() and (q[[1, 2]] == 0).all() and np.isfinite(np.delete(s, [1, 2])).all()


def test_int8_gemm_by_integers():
    rng = np.random.default_rng(3)
    a, b = rng.integers(-128, 128, (5, 64)), rng.integers(-128, 128, (7, 64))
    sa, sb = rng.random(5).astype(np.float32), rng.random(7).astype(np.float32)
    y = int8_gemm_ref(a, sa, b, sb)
    assert y.dtype == np.float32
    for m in range(5):
        for n in range(7):
            total = sum(int(p) * int(q) for p, q in zip(a[m], b[n]))
            assert y[m, n] == np.float32(np.float32(np.float32(total) * sa[m]) * sb[n])


def test_clip():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, c, out = clip_ref(g, 10.0)
    assert norm == 5.0 and c == 1.0 and np.array_equal(out[0], g[0])
    norm, c, out = clip_ref(g, 2.5)
    assert norm == 5.0 and c == 0.5 and np.array_equal(out[1], [[2.0]])
    norm, c, _ = clip_ref([np.array([np.inf])], 1.0)
    assert norm == np.inf and c == 1.0
    assert clip_ref(g, 1.0, norm_sq=100.0)[:2] == (10.0, 0.1)
