"""Rows of the quantized key-value cache on the GPU, bit for bit: codes and scales against oracle/served.py (which takes
the header's fp32 steps), rows read back against the one rounding of code times scale, the fused norm + rotation +
append against its two halves."""
import numpy as np
import pytest

from oracle import served as osv
from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import dev, host
from test_gpu_norm_rope import f64, freqs, make, tdt

pytestmark = pytest.mark.gpu
DIMS = [64, 96, 128, 192, 256]
KINDS = ["int8", "fp4"]
DTYPES = ["fp16", "bf16"]


def oracle_rows(x, kind, dtype):
    """(codes as stored, scales, values) of 16-bit rows [.., D]."""
    if kind == "int8":
        c, s = osv.quant_int8(f64(x))
        return c, s, osv.values_int8(c, s)
    c, s = osv.quant_fp4(f64(x), dtype)
    return osv.pack_fp4(c), s, osv.values_fp4(c, s)


def at_slot(cache, kind, which, page, off):
    """(codes, scales) of one token: [kv, ..]."""
    s = cache[2 + which]
    return host(cache[which][page, :, off]), host(s[page, :, off] if kind == "int8" else s[page, :, :, off])


def check_cache(cache, kind, dtype, k, v, slots, page, fill=0):
    """Every kept token holds its rows; nothing else changed from `fill`."""
    P = cache[0].shape[0]
    kept = {int(s): m for m, s in enumerate(host(slots)) if 0 <= s < P * page}
    for which, x in ((0, k), (1, v)):
        codes, scales, _ = oracle_rows(x, kind, dtype)
        got, gs = host(cache[which]), host(cache[2 + which])
        want, ws = np.full_like(got, fill), np.full_like(gs, fill)
        for s, m in kept.items():
            want[s // page, :, s % page] = codes[m]
            if kind == "int8":
                ws[s // page, :, s % page] = scales[m]
            else:
                ws[s // page, :, :, s % page] = scales[m]
        assert np.array_equal(got, want)
        assert np.array_equal(gs, ws, equal_nan=kind == "int8")


def rows(M, KV, D, dtype, seed=0, special=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, M, KV, D)).astype(np.float32)
    x[:, :, :, rng.integers(0, D, 3)] *= 9
    if special:
        small, big = (2.0 ** -24, 65504.0) if dtype == "fp16" else (2.0 ** -130, 3.0e38)
        for i, row in enumerate([np.zeros(D), np.full(D, small), np.full(D, big), -np.arange(D) * small,
                                 np.where(np.arange(D) == 5, np.inf, 1.0), np.where(np.arange(D) == D - 1, np.nan, 2.0),
                                 np.where(np.arange(D) == 0, -np.inf, 0.0), np.linspace(-6, 6, D),
                                 np.arange(D) * 0.25 - 6, np.where(np.arange(D) < 32, 1e-3, 50.0)]):
            if i < M:
                x[i % 2, i, i % KV] = row
    return [dev(t).to(tdt(dtype)) for t in x]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("KV,D,page", [(1, 64, 16), (3, 96, 32), (8, 128, 16), (2, 192, 64), (5, 256, 16)])
def test_append_and_read(KV, D, page, kind, dtype):
    import torch
    M = 37
    k, v = rows(M, KV, D, dtype, seed=D)
    cache = bd.quant_pages(5, KV, page, D, kind)
    rng = np.random.default_rng(1)
    slots = rng.permutation(5 * page)[:M].astype(np.int64)
    slots[[3, 20]] = [-1, 5 * page]
    slots[11] = -(1 << 40)
    bd.kv_append_quant(k, v, cache, dev(slots))
    check_cache(cache, kind, dtype, k, v, dev(slots), page)
    kept = (slots >= 0) & (slots < 5 * page)
    for out in (dtype, "bf16"):
        if out != dtype and kind == "fp4":
            continue
        back = bd.kv_read_quant(cache, dev(slots), tdt(out))
        for x, got in zip((k, v), back):
            _, _, values = oracle_rows(x, kind, dtype)
            # codes times scales are rounded to fp32 and then to 16 bits, as the kernels do
            with np.errstate(over="ignore"):
                want = torch.from_numpy(values.astype(np.float32)).to(tdt(out)).double().numpy()
            want[~kept] = 0
            assert np.array_equal(f64(got), want, equal_nan=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,H,KV,D,rot,inter", [(1, 8, 1, 256, 256, False), (5, 4, 2, 64, 32, True), (300, 6, 3, 96, 48, True),
                                                (800, 2, 2, 128, 128, False), (2100, 3, 1, 192, 96, False),
                                                (2100, 2, 2, 64, 0, False)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_fused_append_is_its_two_halves(M, H, KV, D, rot, inter, kind, dtype):
    import torch
    q, k, v, wq, wk, pos = make(M, H, KV, D, dtype, seed=M)
    f = freqs(rot)
    f = None if f is None else dev(f)
    page, P = 32, M // 32 + 2
    slots = np.random.default_rng(M).permutation(P * page)[:M].astype(np.int64)
    slots[M // 2] = -1
    slots = dev(slots)
    one, two = (bd.quant_pages(P, KV, page, D, kind) for _ in range(2))
    ko = torch.empty((M, KV, D), dtype=q.dtype, device="cuda")
    qo = bd.qk_norm_rope_append_quant(q, k, v, wq, wk, f, pos, one, slots, interleaved=inter, k_out=ko)
    q2, k2 = bd.qk_norm_rope(q, k, wq, wk, f, pos, interleaved=inter)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    bd.kv_append_quant(k2, v, two, slots)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    if M <= 300:
        check_cache(one, kind, dtype, k2, v, slots, page)
    three = bd.quant_pages(P, KV, page, D, kind)       # without k_out, in place, and without weights
    q3 = q.clone()
    bd.qk_norm_rope_append_quant(q3, k, v, wq, wk, f, pos, three, slots, interleaved=inter, q_out=q3)
    assert torch.equal(q3, qo) and all(torch.equal(a, b) for a, b in zip(one, three))
    bd.qk_norm_rope_append_quant(q, k, v, None, None, f, pos, three, slots, interleaved=inter, k_out=ko)
    bd.kv_append_quant(ko, v, two, slots)
    assert all(torch.equal(a, b) for a, b in zip(two, three))


@pytest.mark.parametrize("kind", KINDS)
def test_row_that_is_not_finite_stays_alone(kind):
    """An infinite channel of one head poisons that head's row (in fp4 its 32 channels) and no other."""
    import torch
    q, k, v, wq, wk, pos = make(9, 2, 2, 128, "fp16", seed=3)
    v = v.clone()
    v[4, 1, 70] = float("inf")
    cache = bd.quant_pages(1, 2, 16, 128, kind)
    slots = torch.arange(9, device="cuda")
    bd.qk_norm_rope_append_quant(q, k, v, wq, wk, dev(freqs(128)), pos, cache, slots)
    _, back = bd.kv_read_quant(cache, slots)
    bad = torch.isnan(back)
    want = torch.zeros_like(bad)
    want[4, 1, slice(64, 96) if kind == "fp4" else slice(None)] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strides_and_neighbours_untouched(kind, offset):
    """Rows that are slices of wider ones at odd addresses; pages, scales and outputs with gaps between them."""
    import torch
    M, KV, D, page, P = 11, 2, 64, 16, 3
    k, v = rows(M, KV, D, "fp16", seed=4)
    wide = torch.full((M, offset + 2 * KV * D + 5), float("nan"), dtype=k.dtype, device="cuda")
    ks, vs = (wide[:, offset + i * KV * D:offset + (i + 1) * KV * D].unflatten(1, (KV, D)) for i in range(2))
    ks.copy_(k), vs.copy_(v)
    slots = dev(np.random.default_rng(2).permutation(P * page)[:M].astype(np.int64))
    small = bd.quant_pages(P, KV, page, D, kind)
    bd.kv_append_quant(k, v, small, slots)
    gap = []
    for t in small:
        big = torch.full((P, t[0].numel() + 32), 7, dtype=t.dtype, device="cuda")
        gap.append((big, big[:, :t[0].numel()].view(t.shape)))
    for _, view in gap:
        view.zero_()
    cache = tuple(view for _, view in gap)
    bd.kv_append_quant(ks, vs, cache, slots)
    for t, (big, view) in zip(small, gap):
        assert torch.equal(host_nan(t), host_nan(view)) and bool((big[:, t[0].numel():] == 7).all())
    out = torch.full((M + 2, offset + KV * D + 3), 9.0, dtype=k.dtype, device="cuda")
    dst = out[:M, offset:offset + KV * D].unflatten(1, (KV, D))
    other = torch.empty_like(k)
    bd.kv_read_quant(cache, slots, k_out=dst, v_out=other)
    want = bd.kv_read_quant(small, slots)
    assert torch.equal(host_nan(dst), host_nan(want[0])) and torch.equal(host_nan(other), host_nan(want[1]))
    out[:M, offset:offset + KV * D] = 9.0
    assert bool((out == 9.0).all())


def host_nan(t):
    import torch
    return torch.nan_to_num(t, nan=1234.0) if t.is_floating_point() else t


@pytest.mark.parametrize("kind", KINDS)
def test_cache_past_32_bits(kind):
    import torch
    KV, D, page = 8, 128, 256
    row = D if kind == "int8" else D // 2
    P = (1 << 32) // (KV * row * page) + 3
    cache = bd.quant_pages(P, KV, page, D, kind)
    k, v = rows(4, KV, D, "bf16", seed=5, special=False)
    slots = dev(np.array([P * page - 1, (P - 2) * page + 17, 5, (P // 2) * page], np.int64))
    bd.kv_append_quant(k, v, cache, slots)
    back = bd.kv_read_quant(cache, slots, torch.bfloat16)
    for i, x in enumerate((k, v)):
        codes, scales, values = oracle_rows(x, kind, "bf16")
        for m, s in enumerate(host(slots)):
            c, e = at_slot(cache, kind, i, s // page, s % page)
            assert np.array_equal(c, codes[m]) and np.array_equal(e, scales[m])
        assert torch.equal(back[i].cpu(), torch.from_numpy(values.astype(np.float32)).bfloat16())


@pytest.mark.parametrize("kind", KINDS)
def test_graph_and_side_stream(kind):
    import torch
    M, H, KV, D = 40, 4, 2, 128
    q, k, v, wq, wk, pos = make(M, H, KV, D, "bf16", seed=6)
    f, slots = dev(freqs(D)), torch.arange(M, device="cuda")
    cache, other = (bd.quant_pages(3, KV, 16, D, kind) for _ in range(2))
    ko, vo, qo = (torch.empty((M, n, D), dtype=q.dtype, device="cuda") for n in (KV, KV, H))

    def call(c):
        bd.qk_norm_rope_append_quant(q, k, v, wq, wk, f, pos, c, slots, q_out=qo)
        bd.kv_read_quant(c, slots, k_out=ko, v_out=vo)
    call(other)
    want = [t.clone() for t in (qo, ko, vo)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(cache)
    for turn in range(4):
        for t in (*cache, qo, ko, vo):
            t.zero_()
        slots.copy_(torch.randperm(48, device="cuda")[:M])
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip((qo, ko, vo), want)), turn
        call(other)
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(other)
        got = [t.clone() for t in (qo, ko, vo)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", KINDS)
def test_empty_and_shared_slots(kind):
    import torch
    k, v = rows(6, 2, 64, "fp16", seed=7, special=False)
    cache = bd.quant_pages(2, 2, 16, 64, kind)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    bd.kv_append_quant(k[:0], v[:0], cache, none)
    assert bd.kv_read_quant(cache, none)[0].shape == (0, 2, 64)
    assert not any(bool(t.any()) for t in cache)
    # rows with one slot that are alike leave that row there; one slot may be read many times
    k[2], v[2], k[4], v[4] = k[0], v[0], k[0], v[0]
    slots = dev(np.array([5, 20, 5, 21, 5, 31], np.int64))
    bd.kv_append_quant(k, v, cache, slots)
    check_cache(cache, kind, "fp16", k, v, slots, 16)
    back = bd.kv_read_quant(cache, slots)[0]
    assert torch.equal(back[0], back[2]) and torch.equal(back[0], back[4])
