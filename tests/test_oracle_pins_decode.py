"""CPU pins of the single-token oracle (oracle/decode.py): closed forms, hand-worked values and
library routines, none of them the device code."""
import numpy as np
import pytest

from oracle import decode as od


def test_pack_w4g_hand_worked():
    W = np.zeros((2, 64), np.float32)
    W[0, :4] = [7.0, -7.0, 3.5, -3.4]      # scale 1: 3.5 is a tie, to the even 4
    W[0, 32:36] = [0.7, -0.05, 0.051, 0.15]
    W[1, 0] = -14.0
    q, s = od.pack_w4g(W, 32)
    assert s.shape == (2, 2) and s[0, 0] == 1.0 and s[0, 1] == 2.0 and s[1, 1] == 1.0
    assert q[0, :4].tolist() == [7, -7, 4, -3]
    assert s[1, 0] == np.float16(np.float32(0.7) / np.float32(7)) and q[0, 32] == 7 and q[0, 34] == 1
    assert q[1, 0] == -7 and not q[1, 1:].any()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack_w4g_rounds_to_nearest(group):
    W = np.random.default_rng(0).normal(0, 0.02, (9, 256)).astype(np.float32)
    q, s = od.pack_w4g(W, group)
    back = q * np.repeat(s.astype(np.float64).T, group, axis=1)
    # half a step, and the largest weight's excess over 7 steps of the rounded scale (2^-11 of 7)
    assert np.all(np.abs(W - back) <= np.repeat(s.astype(np.float64).T, group, axis=1) * (0.5 + 7 * 2.0 ** -10))
    assert np.abs(q).max() == 7


def test_w4g_operand_places_every_code():
    N, K = 18, 160
    codes = np.zeros((N, K), np.int8)
    codes[17, 37] = -3                      # tile (1, 0), row 1, j = 1, g = 0, element 5
    raw = od.w4g_operand(codes)
    assert raw.size == 2 * 2 * 1024
    words = raw.view(np.uint32)
    at = (2 * 1024 + (0 * 16 + 1) * 16 + 4 * 1) // 4
    assert words[at] == (0x88888888 & ~(0xF << 24)) | (5 << 24)  # element 5 is nibble 4 + 5 // 2 = 6
    assert (np.delete(words, at) == 0x88888888).all()


def test_linear_w4g_matches_a_loop():
    rng = np.random.default_rng(1)
    X, W = rng.standard_normal((3, 64)), rng.normal(0, 1, (5, 64)).astype(np.float32)
    q, s = od.pack_w4g(W, 32)
    y, size = od.linear_w4g(X, q, s)
    for m in range(3):
        for n in range(5):
            t = [X[m, k] * float(q[n, k]) * float(s[k // 32, n]) for k in range(64)]
            assert abs(y[m, n] - sum(t)) < 1e-12 and abs(size[m, n] - sum(map(abs, t))) < 1e-12
    g, _ = od.linear_w4g(X, q, s, "gelu")
    from math import erf, sqrt
    assert abs(g[1, 2] - 0.5 * y[1, 2] * (1 + erf(y[1, 2] / sqrt(2)))) < 1e-12


def test_norm_rope_hand_worked():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y = od.norm_rope(x, None, 0.0, None, None, False)          # mean square 25 / 4
    assert np.allclose(y, [[[1.2, 1.6, 0, 0]]], atol=1e-15)
    quarter = np.array([np.pi / 2, 0.0])
    half = od.norm_rope(x, None, 0.0, quarter, [1], False)     # pairs (0, 2), (1, 3): only the first turns
    assert np.allclose(half, [[[0, 1.6, 1.2, 0]]], atol=1e-15)
    pair = od.norm_rope(x, None, 0.0, quarter, [1], True)      # pairs (0, 1), (2, 3)
    assert np.allclose(pair, [[[-1.6, 1.2, 0, 0]]], atol=1e-15)
    part = od.norm_rope(x, np.array([1, 2, 3, 4.0]), 0.0, quarter[:1], [2], True)
    assert np.allclose(part, [[[-1.2, -3.2, 0, 0]]], atol=1e-15)


def test_norm_rope_keeps_length_and_relative_angle():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 32))
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    rot = lambda x, p: od.norm_rope(x, None, 0.0, f, [p], False)[0, 0]  # noqa: E731
    assert np.allclose(np.linalg.norm(rot(q, 1234)), np.sqrt(32))
    # the product of a rotated query and key depends on the distance alone
    assert abs(rot(q, 107) @ rot(k, 100) - rot(q, 7) @ rot(k, 0)) < 1e-10


def test_append_skips_and_places():
    c = od.append(np.zeros((2, 1, 4, 2)), np.arange(10.0).reshape(5, 1, 2), [5, -1, 0, 8, 1 << 40])
    assert c[1, 0, 1].tolist() == [0, 1] and c[0, 0, 0].tolist() == [4, 5] and np.count_nonzero(c) == 3


def test_paged_attention_matches_dense_softmax():
    from scipy.special import softmax
    rng = np.random.default_rng(3)
    page, n, D = 4, 10, 8
    keys, vals, q = rng.standard_normal((n, 1, D)), rng.standard_normal((n, 1, D)), rng.standard_normal((1, 2, D))
    table = np.array([[4, 0, 2, -1]], np.int32)
    kc, vc = np.full((5, 1, page, D), np.nan), np.full((5, 1, page, D), np.nan)
    for j in range(n):
        kc[table[0, j // page], 0, j % page], vc[table[0, j // page], 0, j % page] = keys[j, 0], vals[j, 0]
    for window, sinks, js in ((0, 0, range(10)), (3, 0, (7, 8, 9)), (3, 2, (0, 1, 7, 8, 9)), (9, 5, range(10))):
        js = list(js)
        got = od.paged_attention(q, kc, vc, table, [n], 0.3, window, sinks)
        for h in range(2):
            want = softmax(keys[js, 0] @ q[0, h] * 0.3) @ vals[js, 0]
            assert np.allclose(got[0, h], want, atol=1e-14), (window, sinks)


def test_paged_attention_empty_and_bad():
    q, kc = np.ones((4, 1, 2)), np.ones((1, 1, 4, 2))
    table = np.array([[0], [0], [3], [-1]], np.int32)
    out = od.paged_attention(q, kc, kc, table, [0, 5, 2, 1], 1.0)
    assert (out[0] == 0).all() and np.isnan(out[1:]).all()
