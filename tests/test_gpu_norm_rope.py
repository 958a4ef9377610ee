"""GPU parity of the per-head norm + position rotation (+ cache append) against the fp64 oracle.

Tolerance from the arithmetic, u = 2^-24: the sum of squares adds at most 8 + 6 terms deep, its error is
halved by the root, rsqrt is within 2 units and three products follow, so a normalized value is within
32 u. The angle in turns carries |t| 2^-51 (three fp64 roundings, here and in the oracle), its fraction
is rounded to fp32 (2^-26 turns) and sine and cosine are within 2 units of fp32: 2^-22 in all. A
rotated channel is then within (|a| + |b|) (34 u + 2^-22 + |t| 2^-51), and rounded once."""
import numpy as np
import pytest

from oracle import decode as od
from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import dev, host

pytestmark = pytest.mark.gpu
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def tdt(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}[name]


def f64(t):
    return host(t.double())


def freqs(rot):
    return 10000.0 ** (-np.arange(0, rot, 2) / rot) if rot else None


def make(M, H, KV, D, dtype, seed=0, scale=2.0):
    import torch
    rng = np.random.default_rng(seed)
    qkv = dev((rng.standard_normal((M, (H + 2 * KV) * D)) * scale).astype(np.float32)).to(tdt(dtype))
    q = qkv[:, :H * D].view(M, H, D)
    k = qkv[:, H * D:(H + KV) * D].view(M, KV, D)
    v = qkv[:, (H + KV) * D:].view(M, KV, D)
    w = [dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2)]
    pos = dev(rng.integers(0, 1 << 20, M).astype(np.int64))
    assert torch.cuda.is_available()
    return q, k, v, w[0], w[1], pos


def check(got, x, w, eps, inv_freq, pos, interleaved, dtype):
    want = od.norm_rope(f64(x), None if w is None else host(w), eps, inv_freq, host(pos), interleaved)
    plain = np.abs(od.norm_rope(f64(x), None if w is None else host(w), eps, None, None, False))
    half = 0 if inv_freq is None else len(inv_freq)
    both = plain.copy()
    rel = np.full(plain.shape, 34 * 2.0 ** -24)
    if half:
        ia = np.arange(half) * 2 if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        s = plain[..., ia] + plain[..., ib]
        both[..., ia], both[..., ib] = s, s
        t = np.abs(host(pos).astype(np.float64)[:, None] * inv_freq)[:, None, :] * 2.0 ** -51 + 2.0 ** -22
        rel[..., ia] += t
        rel[..., ib] += t
    tol = both * rel
    tol = tol + HALF_STEP[dtype] * (np.abs(want) + tol) + 2.0 ** -25
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:5])


SHAPES = [(1, 8, 1, 256, 256), (1, 1, 1, 16, 16), (5, 3, 2, 64, 64), (7, 16, 16, 64, 32), (33, 5, 1, 96, 96),
          (3, 4, 4, 128, 0), (9, 6, 2, 192, 128), (2, 2, 1, 80, 80), (4, 2, 2, 512, 512), (50, 32, 8, 128, 128),
          (1500, 4, 2, 32, 32), (6, 2, 2, 112, 16)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M,H,KV,D,rot", SHAPES)
def test_norm_rope(M, H, KV, D, rot, interleaved, dtype):
    q, k, _, wq, wk, pos = make(M, H, KV, D, dtype, seed=D + M)
    f = freqs(rot)
    fd = None if f is None else dev(f)
    qo, ko = bd.qk_norm_rope(q, k, wq, wk, fd, pos if rot else None, 1e-6, interleaved)
    check(qo, q, wq, 1e-6, f, pos, interleaved, dtype)
    check(ko, k, wk, 1e-6, f, pos, interleaved, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,H,KV,D,page,pad", [(1, 8, 1, 256, 16, 0), (41, 4, 2, 64, 16, 3), (1100, 2, 2, 96, 64, 9),
                                                (20, 3, 1, 128, 4096, 1)])
def test_append(M, H, KV, D, page, pad, dtype):
    import torch
    q, k, v, wq, wk, pos = make(M, H, KV, D, dtype, seed=M)
    f = freqs(D)
    P = -(-M // page) + 2
    rng = np.random.default_rng(5)
    slots = rng.permutation(P * page)[:M].astype(np.int64)
    slots[M - pad:] = -1
    if pad > 1:
        slots[M - 2] = P * page          # past the cache: skipped
    if pad > 2:
        slots[M - 3] = 1 << 40
    kc = torch.full((P, KV, page, D), 5.0, dtype=q.dtype, device="cuda")
    vc = torch.full((P, KV, page, D), 6.0, dtype=q.dtype, device="cuda")
    before = q.clone(), k.clone(), v.clone()
    ko = torch.empty_like(k)
    qo = bd.qk_norm_rope_append(q, k, v, wq, wk, dev(f), pos, kc, vc, dev(slots), k_out=ko)
    check(qo, q, wq, 1e-6, f, pos, False, dtype)
    check(ko, k, wk, 1e-6, f, pos, False, dtype)
    # the cache holds exactly those rows, and nothing else changed
    assert np.array_equal(f64(kc), od.append(np.full(kc.shape, 5.0), f64(ko), slots))
    assert np.array_equal(f64(vc), od.append(np.full(vc.shape, 6.0), f64(v), slots))
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, v)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [3, 1200])
def test_in_place_strides_and_no_weights(M, dtype):
    """In place on slices of a QKV buffer with odd row strides; what is around them stays."""
    import torch
    H, KV, D = 4, 2, 64
    q, k, _, _, _, pos = make(M, H, KV, D, dtype, seed=8)
    buf = torch.full((M, 1 + (H + KV) * D + 2), 3.0, dtype=q.dtype, device="cuda")
    buf[:, 1:1 + H * D] = q.reshape(M, -1)
    buf[:, 1 + H * D:1 + (H + KV) * D] = k.reshape(M, -1)
    qs = buf[:, 1:1 + H * D].unflatten(1, (H, D))
    ks = buf[:, 1 + H * D:1 + (H + KV) * D].unflatten(1, (KV, D))
    f = freqs(D)
    bd.qk_norm_rope(qs, ks, None, None, dev(f), pos, 1e-5, False, q_out=qs, k_out=ks)
    check(qs, q, None, 1e-5, f, pos, False, dtype)
    check(ks, k, None, 1e-5, f, pos, False, dtype)
    assert bool((buf[:, 0] == 3).all()) and bool((buf[:, -2:] == 3).all())


def test_far_positions():
    import torch
    q, k, _, wq, wk, _ = make(6, 2, 1, 128, "bf16", seed=3)
    pos = torch.tensor([0, 1, (1 << 20) + 1, (1 << 31) - 1, 1 << 31, (1 << 33) + 12345], device="cuda")
    f = freqs(128)
    qo, ko = bd.qk_norm_rope(q, k, wq, wk, dev(f), pos)
    check(qo, q, wq, 1e-6, f, pos, False, "bf16")
    check(ko, k, wk, 1e-6, f, pos, False, "bf16")


def test_zero_small_and_non_finite_heads():
    """A head of zeros stays zero, subnormal heads are normalized, a NaN or infinity stays in its head."""
    import torch
    q, k, _, wq, wk, pos = make(4, 3, 1, 64, "fp16", seed=4)
    q[0, 0] = 0
    q[1, 1] = 2.0 ** -24
    q[2, 2, 7] = float("nan")
    q[3, 0, 1] = float("inf")
    f = freqs(32)
    qo, _ = bd.qk_norm_rope(q, k, wq, wk, dev(f), pos, 1e-12)
    assert bool((qo[0, 0] == 0).all())
    assert bool(torch.isnan(qo[2, 2]).all())
    assert bool(torch.isnan(qo[3, 0, 1]).all())
    keep = torch.ones(4, 3, dtype=torch.bool)
    keep[2, 2] = keep[3, 0] = False
    for m in range(4):
        heads = [h for h in range(3) if keep[m, h]]
        check(qo[m:m + 1, heads], q[m:m + 1, heads], wq, 1e-12, f, pos[m:m + 1], False, "fp16")


def test_slots_past_32_bits():
    """Rows that land beyond 2^31 elements of the cache."""
    import torch
    KV, D, page = 8, 128, 256
    P = (1 << 31) // (KV * D * page) + 3
    q, k, v, wq, wk, pos = make(2, 2, KV, D, "fp16", seed=6)
    kc = torch.empty((P, KV, page, D), dtype=torch.float16, device="cuda")
    vc = torch.empty((P, KV, page, D), dtype=torch.float16, device="cuda")
    slots = torch.tensor([P * page - 1, (P - 2) * page + 3], device="cuda")
    ko = torch.empty_like(k)
    bd.qk_norm_rope_append(q, k, v, wq, wk, dev(freqs(D)), pos, kc, vc, slots, k_out=ko)
    assert torch.equal(kc[P - 1, :, page - 1], ko[0]) and torch.equal(vc[P - 1, :, page - 1], v[0])
    assert torch.equal(kc[P - 2, :, 3], ko[1]) and torch.equal(vc[P - 2, :, 3], v[1])


def test_graph_replays_and_side_stream():
    import torch
    q, k, v, wq, wk, pos = make(5, 4, 2, 64, "bf16", seed=7)
    f = dev(freqs(64))
    kc = torch.zeros((3, 2, 16, 64), dtype=q.dtype, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.arange(5, device="cuda")
    qo = torch.empty_like(q)
    run = lambda: bd.qk_norm_rope_append(q, k, v, wq, wk, f, pos, kc, vc, slots, q_out=qo)  # noqa: E731
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        pos += 11
        slots += 7
        kc.zero_()
        vc.zero_()
        graph.replay()
        got = qo.clone(), kc.clone(), vc.clone()
        kc.zero_()
        vc.zero_()
        run()
        assert all(torch.equal(a, b) for a, b in zip(got, (qo, kc, vc))), i
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = bd.qk_norm_rope(q, k, wq, wk, f, pos)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, qo)


def test_empty_batch():
    q, k, v, wq, wk, pos = make(2, 2, 1, 64, "fp16")
    qo, ko = bd.qk_norm_rope(q[:0], k[:0], wq, wk, dev(freqs(64)), pos[:0])
    assert qo.shape == (0, 2, 64) and ko.shape == (0, 1, 64)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 32), (96, 16), (64, 0), (128, 128)])
def test_infinity_stays_in_its_pair(D, rot, interleaved, dtype):
    """An infinite channel makes its head's mean infinite: every other channel is 0, the channel itself and,
    where it is rotated, the other one of its pair are NaN. Neighbours that are not rotated are no pair."""
    import torch
    q, k, _, wq, wk, pos = make(D, 2, 1, D, dtype, seed=D + rot)
    f = freqs(rot)
    for m in range(D):
        q[m, 0, m] = float("inf") if m % 2 else float("-inf")
        k[m, 0, D - 1 - m] = float("inf")
    qo, ko = bd.qk_norm_rope(q, k, wq, wk, None if f is None else dev(f), pos if rot else None, 1e-6, interleaved)
    for got, x, w in ((qo[:, :1], q[:, :1], wq), (ko, k, wk)):
        with np.errstate(invalid="ignore"):
            want = od.norm_rope(f64(x), host(w), 1e-6, f, host(pos), interleaved)
        assert np.array_equal(f64(got), want, equal_nan=True), np.argwhere(np.isnan(f64(got)) != np.isnan(want))[:5]
    assert torch.isfinite(qo[:, 1]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("M", [399, 500, 801, 1400, 1700, 3300])
def test_any_number_of_waves_per_token(M, interleaved, dtype):
    """From eight waves on a token to four tokens in a workgroup: against the oracle, and a token's values do not
    depend on how many others there are."""
    import torch
    H, KV, D = 9, 3, 64
    q, k, v, wq, wk, pos = make(M, H, KV, D, dtype, seed=M)
    f = freqs(32)
    page = 16
    P = -(-M // page) + 1
    slots = np.random.default_rng(M).permutation(P * page)[:M].astype(np.int64)
    slots[M // 2] = -1
    kc, vc = (torch.full((P, KV, page, D), 5.0, dtype=q.dtype, device="cuda") for _ in range(2))
    ko = torch.empty_like(k)
    qo = bd.qk_norm_rope_append(q, k, v, wq, wk, dev(f), pos, kc, vc, dev(slots), interleaved=interleaved, k_out=ko)
    check(qo, q, wq, 1e-6, f, pos, interleaved, dtype)
    check(ko, k, wk, 1e-6, f, pos, interleaved, dtype)
    assert np.array_equal(f64(kc), od.append(np.full(kc.shape, 5.0), f64(ko), slots))
    assert np.array_equal(f64(vc), od.append(np.full(vc.shape, 5.0), f64(v), slots))
    for a in (0, M - 7):
        qa, ka = bd.qk_norm_rope(q[a:a + 7], k[a:a + 7], wq, wk, dev(f), pos[a:a + 7], interleaved=interleaved)
        assert torch.equal(qa, qo[a:a + 7]) and torch.equal(ka, ko[a:a + 7])
