"""Plain CPU oracle (numpy) of the quantized key-value cache's rows, the attention behind a shared prefix and the
low-rank adapters of many requests. Written from the definitions in include/w4a4.h; shares no code with the device
path. Codes and scales follow the header's fp32 steps bit for bit, everything else is fp64."""
from __future__ import annotations

import numpy as np

from . import decode as od

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FP4_RANGE = {"fp16": (-23, 13), "bf16": (-100, 125)}


# ---- rows of the quantized cache -----------------------------------------------------------------

def quant_int8(x):
    """Rows x [..., D] of 16-bit values: (codes int8 [..., D], scale fp32 [...])."""
    x = np.asarray(x, np.float32)
    m = np.abs(x).max(-1)
    with np.errstate(invalid="ignore", over="ignore"):
        mm = np.maximum(m, np.float32(2.0 ** -100))
        s = (mm / np.float32(127)).astype(np.float32)
        r = (np.float32(127) / mm).astype(np.float32)
        t = np.rint((x * r[..., None]).astype(np.float32))
    ok = np.isfinite(m)
    return (np.where(ok[..., None], np.nan_to_num(t, nan=0.0), 0).astype(np.int8),
            np.where(ok, s, np.float32("nan")).astype(np.float32))


def quant_fp4(x, dtype):
    """Rows x [..., D]: (E2M1 codes uint8 [..., D] one per entry, exponent bytes uint8 [..., D / 32])."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, 32)
    m = np.abs(g).max(-1)
    ok = np.isfinite(m)
    lo, hi = FP4_RANGE[dtype]
    e = np.full(m.shape, lo, np.int64)
    for n in range(lo, hi):               # the smallest that holds m, by trying
        e = np.where(np.where(ok, m, 0.0) > 6.0 * 2.0 ** e.astype(np.float64), n + 1, e)
    with np.errstate(invalid="ignore"):
        y = np.abs(g) / 2.0 ** e.astype(np.float64)[..., None]
    y = np.where(np.isfinite(y), np.minimum(y, 6.0), 0.0)
    d = np.abs(y[..., None] - E2M1)
    near = d == d.min(-1, keepdims=True)
    # of two equally near ones the even code
    code = np.where(near.sum(-1) > 1, np.where(near & (np.arange(8) % 2 == 0), np.arange(8), -1).max(-1), d.argmin(-1))
    code = code | (np.signbit(g) << 3)
    code = np.where(ok[..., None], code, 0).astype(np.uint8)
    return code.reshape(x.shape), np.where(ok, e + 127, 255).astype(np.uint8)


def pack_fp4(codes):
    """Two codes per byte, the even channel low."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values_int8(codes, scale):
    return codes.astype(np.float64) * scale.astype(np.float64)[..., None]


def values_fp4(codes, scale):
    """codes one per entry [..., D], scale bytes [..., D / 32]."""
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)


# ---- attention behind a shared prefix ----------------------------------------------------------------

def shared_attention(q, k_cache, v_cache, prefix_table, prefix_len, table, lens, scale):
    """Caches are fp64 values [pages, kv_heads, page, D]. The sequences are put together page by page and token by
    token, and attended to as any other."""
    B, H, D = q.shape
    P, KV, page, _ = k_cache.shape
    out = np.zeros((B, H, D))

    def tokens(row, n):
        j = np.arange(max(n, 0))
        if j.size and j[-1] // page >= len(row):
            return None
        ids = np.asarray(row)[j // page].astype(np.int64)
        if ((ids < 0) | (ids >= P)).any():
            return None
        return ids, j % page

    first = tokens(prefix_table, prefix_len)
    for b in range(B):
        own = tokens(table[b], int(lens[b]))
        if first is None or own is None:
            out[b] = np.nan
            continue
        ids, off = (np.concatenate([x, y]) for x, y in zip(first, own))
        if not ids.size:
            continue
        for h in range(H):
            k, v = k_cache[ids, h * KV // H, off], v_cache[ids, h * KV // H, off]
            s = k @ np.asarray(q[b, h], np.float64) * scale
            p = np.exp(s - s.max())
            out[b, h] = (p / p.sum()) @ v
    return out


# ---- low-rank adapters --------------------------------------------------------------------------------

def adapter_add(Y, X, A, B, ids, scale=None, epilogue="none", residual=None):
    """fp64 result, and the sizes that its error is made of: per output sum_r |b| (sum_k |x||a|) and sum_r |b||t|,
    both times |scale|, and the sum before the epilogue."""
    Y, X, A, B = (np.asarray(t, np.float64) for t in (Y, X, A, B))
    y = Y.copy()
    inner, outer = np.zeros_like(Y), np.zeros_like(Y)
    for m, a in enumerate(ids):
        if not 0 <= a < len(A):
            continue
        s = 1.0 if scale is None else float(scale[a])
        t = A[a] @ X[m]
        y[m] += s * (B[a] @ t)
        inner[m] = abs(s) * (np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(X[m])))
        outer[m] = abs(s) * (np.abs(B[a]) @ np.abs(t))
    pre = y.copy()
    if epilogue == "gelu":
        y = y * od.ndtr(y)
    elif epilogue == "residual":
        y = y + np.asarray(residual, np.float64)
    return y, inner, outer, pre
