"""CPU pins of oracle/served.py: closed forms, hand-worked values and other ways to the same numbers, none of them
the device code."""
import numpy as np
import pytest

from oracle import decode as od
from oracle import served as osv


def test_int8_rows_hand_worked():
    x = np.zeros((3, 64), np.float32)
    x[0, :5] = [127.0, -127.0, 0.5, 1.5, -2.5]       # scale 1: halves go to even
    x[1, 0] = -254.0
    c, s = osv.quant_int8(x)
    assert c[0, :5].tolist() == [127, -127, 0, 2, -2] and s[0] == 1.0
    assert c[1, 0] == -127 and s[1] == 2.0 and not c[2].any()
    assert osv.values_int8(c, s)[2].max() == 0.0 and np.isfinite(s[2])


def test_int8_rounds_to_nearest():
    x = np.random.default_rng(0).standard_normal((50, 128)).astype(np.float16).astype(np.float32)
    c, s = osv.quant_int8(x)
    assert np.all(np.abs(osv.values_int8(c, s) - x) <= s[:, None] * (0.5 + 127 * 2.0 ** -22))
    assert np.all(np.abs(c).max(-1) == 127)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_rows_that_are_not_finite(bad):
    x = np.ones((2, 64))
    x[0, 40] = bad
    c, s = osv.quant_int8(x)
    assert np.isnan(s[0]) and not c[0].any() and np.isfinite(s[1])
    c, e = osv.quant_fp4(x, "fp16")
    assert e.tolist()[0][1] == 255 and e[0, 0] != 255 and not c[0, 32:].any()
    v = osv.values_fp4(c, e)
    assert np.isnan(v[0, 32:]).all() and np.array_equal(v[0, :32], np.ones(32)) and np.array_equal(v[1], np.ones(64))


def test_fp4_hand_worked():
    x = np.zeros((1, 64))
    x[0, :10] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.5]     # scale 1, all the ties
    x[0, 32:35] = [6.0001, 3.0, -6.0]                                          # scale 2
    c, e = osv.quant_fp4(x, "fp16")
    assert e[0].tolist() == [127, 128]
    assert c[0, :10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 15]
    assert osv.values_fp4(c, e)[0, 32:35].tolist() == [6.0, 3.0, -6.0]
    assert osv.pack_fp4(c)[0, :2].tolist() == [7 | 0 << 4, 2 | 2 << 4]


@pytest.mark.parametrize("dtype,lo,hi", [("fp16", -23, 13), ("bf16", -100, 125)])
def test_fp4_scale_stays_in_its_range(dtype, lo, hi):
    x = np.zeros((2, 32))
    x[0, 0] = 2.0 ** (lo - 2)
    x[1, :2] = [6.5 * 2.0 ** hi, -2.0 ** hi]
    c, e = osv.quant_fp4(x, dtype)
    assert e[:, 0].tolist() == [lo + 127, hi + 127]
    assert c[0, 0] == 0 and c[1, 0] == 7 and osv.values_fp4(c, e)[1, 1] == -2.0 ** hi


def test_fp4_is_the_nearest_value():
    x = np.random.default_rng(1).standard_normal((40, 96)).astype(np.float32).astype(np.float64)
    c, e = osv.quant_fp4(x, "bf16")
    v = osv.values_fp4(c, e)
    grid = np.concatenate([osv.E2M1, -osv.E2M1])
    s = np.repeat(2.0 ** (e.astype(np.float64) - 127), 32, -1)
    best = np.abs(x[..., None] - grid * s[..., None]).min(-1)
    assert np.allclose(np.abs(x - v), best, rtol=0, atol=1e-15)
    assert np.all(np.abs(x).reshape(40, 3, 32).max(-1) > 3.0 * 2.0 ** (e.astype(np.float64) - 127))


def test_shared_attention_is_attention_over_the_joined_pages():
    rng = np.random.default_rng(2)
    q = rng.standard_normal((3, 4, 64))
    k, v = rng.standard_normal((2, 12, 2, 16, 64))
    prefix, table = np.array([3, 7]), np.array([[0, 1], [2, 4], [5, 6]])
    got = osv.shared_attention(q, k, v, prefix, 32, table, [20, 0, 7], 0.2)
    want = od.paged_attention(q, k, v, np.concatenate([np.tile(prefix, (3, 1)), table], 1), [52, 32, 39], 0.2)
    assert np.allclose(got, want, rtol=1e-13, atol=1e-15)
    assert not osv.shared_attention(q, k, v, prefix, 0, table, [0, 0, 0], 0.2).any()
    assert np.isnan(osv.shared_attention(q, k, v, prefix, 33, table, [0, 0, 1], 0.2)).all()


def test_adapters_are_weights_added():
    rng = np.random.default_rng(3)
    X, W = rng.standard_normal((5, 24)), rng.standard_normal((7, 24))
    A, B = rng.standard_normal((2, 8, 24)), rng.standard_normal((2, 7, 8))
    ids, s = [1, -1, 0, 2, 1], np.array([0.5, -2.0])
    y = osv.adapter_add(X @ W.T, X, A, B, ids, s)[0]
    for m, a in enumerate(ids):
        full = W if a not in (0, 1) else W + s[a] * (B[a] @ A[a])
        assert np.allclose(y[m], full @ X[m], rtol=1e-12)
    r = rng.standard_normal((5, 7))
    assert np.allclose(osv.adapter_add(X @ W.T, X, A, B, ids, s, "residual", r)[0], y + r)
    g = osv.adapter_add(X @ W.T, X, A, B, ids, s, "gelu")[0]
    from scipy.special import erf
    assert np.allclose(g, 0.5 * y * (1 + erf(y / np.sqrt(2))), rtol=1e-9, atol=1e-12)
