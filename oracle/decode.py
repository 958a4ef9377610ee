"""Plain CPU oracle of the single-token operators (numpy, fp64): linears with group-scaled 4-bit
weights, the per-head norm and position rotation with the append to a paged cache, and the attention
of one new token per sequence over that cache. Written from the definitions in include/w4a4.h; shares
no code with the device path."""
from __future__ import annotations

import numpy as np
from scipy.special import ndtr


# ---- group-scaled 4-bit linears ---------------------------------------------------------------

def pack_w4g(W, group: int):
    """Round to nearest per group. Returns (codes int8 [N, K], scale fp16 [K / group, N])."""
    W = np.asarray(W, np.float32)
    N, K = W.shape
    g = W.reshape(N, K // group, group)
    mx = np.abs(g).max(-1)
    s = np.minimum(mx / np.float32(7), np.float32(65504)).astype(np.float16)
    s = np.where(s == 0, np.where(mx == 0, np.float16(1), np.float16(2.0 ** -24)), s)
    q = np.rint(g / s.astype(np.float32)[..., None])
    return np.clip(q, -8, 7).astype(np.int8).reshape(N, K), np.ascontiguousarray(s.T)


def w4g_operand(codes):
    """The tiled operand bytes of codes [N, K], dword by dword as the header lays them out."""
    N, K = codes.shape
    n16, k128 = -(-N // 16), -(-K // 128)
    full = np.zeros((n16 * 16, k128 * 128), np.int64)
    full[:N, :K] = codes
    out = np.zeros(n16 * k128 * 256, np.uint32)
    for n in range(n16 * 16):
        for k0 in range(0, k128 * 128, 8):
            word = 0
            for i in range(8):
                e = 2 * i if i < 4 else 2 * (i - 4) + 1
                word |= int(full[n, k0 + e] + 8) << (4 * i)
            j, g = (k0 % 128) // 32, (k0 % 32) // 8
            byte = ((n // 16) * k128 + k0 // 128) * 1024 + (g * 16 + n % 16) * 16 + 4 * j
            out[byte // 4] = word
    return out.view(np.uint8)


def linear_w4g(X, codes, scale, epilogue: str = "none", residual=None):
    """fp64 result, and sum |x| |c| s per output (the size its fp32 sums are made of)."""
    X = np.asarray(X, np.float64)
    group = codes.shape[1] // scale.shape[0]
    W = codes.astype(np.float64) * np.repeat(scale.astype(np.float64).T, group, axis=1)
    with np.errstate(invalid="ignore", over="ignore"):
        y, size = X @ W.T, np.abs(X) @ np.abs(W).T
    if epilogue == "gelu":
        y = y * ndtr(y)
    elif epilogue == "residual":
        y = y + np.asarray(residual, np.float64)
    return y, size


# ---- norm, rotation, append -------------------------------------------------------------------

def norm_rope(x, weight, eps, inv_freq, positions, interleaved: bool):
    """x [M, heads, D]: per-head RMS norm, then the first 2 * len(inv_freq) channels rotated in pairs
    by position * inv_freq."""
    x = np.asarray(x, np.float64)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    half = 0 if inv_freq is None else len(inv_freq)
    if half:
        t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
        c, s = np.cos(t)[:, None, :], np.sin(t)[:, None, :]
        ia = np.arange(half) * 2 if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def append(cache, rows, slots):
    """rows [M, kv_heads, D] into cache [pages, kv_heads, page, D] at slots (page * page_size + offset);
    a slot outside the cache is skipped."""
    out = np.array(cache)
    P, _, page, _ = out.shape
    for m, s in enumerate(slots):
        if 0 <= s < P * page:
            out[s // page, :, s % page] = rows[m]
    return out


# ---- attention over the cache -----------------------------------------------------------------

def visible(n: int, window: int, sinks: int):
    j = np.arange(max(n, 0))
    return j if window <= 0 else j[(j < sinks) | (j >= n - window)]


def paged_attention(q, k_cache, v_cache, table, lens, scale, window: int = 0, sinks: int = 0):
    """q [B, heads, D]; returns fp64 [B, heads, D] (zeros where nothing is visible; NaN where a visible
    page's entry does not name a page)."""
    q = np.asarray(q, np.float64)
    B, H, D = q.shape
    P, KV, page, _ = k_cache.shape
    out = np.zeros((B, H, D))
    for b in range(B):
        j = visible(int(lens[b]), window, sinks)
        if j.size == 0:
            continue
        if j[-1] // page >= table.shape[1]:
            out[b] = np.nan
            continue
        ids = table[b, j // page].astype(np.int64)
        if ((ids < 0) | (ids >= P)).any():
            out[b] = np.nan
            continue
        for h in range(H):
            k = k_cache[ids, h * KV // H, j % page].astype(np.float64)
            v = v_cache[ids, h * KV // H, j % page].astype(np.float64)
            s = k @ q[b, h] * scale
            p = np.exp(s - s.max())
            out[b, h] = (p / p.sum()) @ v
    return out
