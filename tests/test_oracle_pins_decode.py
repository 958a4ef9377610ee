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
