"""GPU parity of the linears with group-scaled 4-bit weights against the fp64 oracle.

Tolerance, per output, from the arithmetic: the products of a code and an activation are exact (fp32
activations in three parts, so three products); a sum of n terms in fp32 of any order is off by at
most n u S with S = sum |x||c|s and u = 2^-23 (one whole unit per step, in case the matrix cores cut
instead of rounding); each group adds one FMA and the scale's product with S, the workgroup's join one
addition per wave. The epilogue then rounds once to fp16 (half a step: 2^-11 relative, 2^-25 for
subnormals) or bf16 (2^-8). GELU has slope at most 1.13, and its own evaluation is within 2^-15
relative (the rounded argument moves erfc by 2 z^2 2^-24 relative, z < 10, plus a few units)."""
import numpy as np
import pytest

from oracle import decode as od
from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import dev, host

pytestmark = pytest.mark.gpu

EPIS = {"none": bd.EPI_NONE, "gelu": bd.EPI_GELU, "residual": bd.EPI_RESIDUAL}
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -11}


def tdt(name):
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def out_dt(name):
    return tdt("bf16") if name == "bf16" else tdt("fp16")


def f64(t):
    return host(t.double())


def make(M, K, N, group, dtype, seed=0):
    rng = np.random.default_rng(seed)
    W = rng.normal(0, 0.02, (N, K)).astype(np.float32)
    W[rng.integers(0, N, 1)] *= 10
    X = rng.standard_normal((M, K)).astype(np.float32)
    X[:, rng.integers(0, K, max(1, K // 100))] *= 20
    codes, s = od.pack_w4g(W, group)
    return W, dev(X).to(tdt(dtype)), codes, s


def tolerance(y, size, K, group, dtype, epi):
    parts = 3 if dtype == "fp32" else 1
    acc = (parts * K + 3 * (K // group) + 32) * 2.0 ** -23 * size
    t = acc
    if epi == "gelu":
        t = 1.13 * acc + 2.0 ** -15 * np.abs(y)
    elif epi == "residual":
        t = acc + 2.0 ** -23 * np.abs(y)
    return t + HALF_STEP[dtype] * (np.abs(y) + t) + 2.0 ** -25


def check(Y, X, codes, s, group, dtype, epi="none", residual=None):
    y, size = od.linear_w4g(f64(X), codes, s, epi, None if residual is None else f64(residual))
    err = np.abs(f64(Y) - y)
    tol = tolerance(y, size, codes.shape[1], group, dtype, epi)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:5])


CASES = [(1, 32, 1, 32), (1, 256, 16, 64), (1, 1024, 100, 128), (3, 96, 5, 32), (16, 256, 256, 64),
         (17, 160, 33, 32), (2, 512, 31, 256), (33, 512, 100, 256), (50, 1024, 130, 128),
         (64, 2048, 48, 64), (65, 256, 40, 128), (130, 384, 17, 128), (5, 16384, 35, 128),
         (1, 192, 47, 64), (48, 4096, 20, 32)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,K,N,group", CASES)
def test_linear(M, K, N, group, dtype):
    _, X, codes, s = make(M, K, N, group, dtype, seed=M + K)
    wt, sd = dev(od.w4g_operand(codes)), dev(s)
    res = dev(np.random.default_rng(1).standard_normal((M, N)).astype(np.float32)).to(out_dt(dtype))
    for epi, code in EPIS.items():
        r = res if epi == "residual" else None
        check(bd.gemv_w4g(X, wt, sd, epilogue=code, residual=r), X, codes, s, group, dtype, epi, r)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("N,K,group", [(16, 256, 64), (1, 32, 32), (37, 416, 32), (18, 768, 256), (33, 384, 128)])
def test_pack_matches_oracle(N, K, group, dtype):
    rng = np.random.default_rng(3)
    W = rng.normal(0, 0.02, (N, K)).astype(np.float32)
    W[0, :group] = 0                       # a group of zeros
    if N > 1:
        W[1, :group] *= 1e-6               # scale below fp16's smallest: held at 2^-24
    if dtype != "fp16" and N > 2:
        W[2, :group] *= 1e9                # scale above fp16's largest: held at 65504
    Wd = dev(W).to(tdt(dtype))
    W32 = host(Wd.float())
    codes, s = od.pack_w4g(W32, group)
    wt, sd = bd.pack_weights_w4g(Wd, group)
    assert np.array_equal(host(sd), s)
    assert np.array_equal(host(wt), od.w4g_operand(codes))
    packed = dev((codes[:, 0::2] & 15 | (codes[:, 1::2] & 15) << 4).astype(np.uint8))
    assert np.array_equal(host(bd.codes_to_w4g(packed, K)), od.w4g_operand(codes))


def test_pack_strided_rows():
    rng = np.random.default_rng(4)
    W = dev(rng.normal(0, 0.02, (20, 300)).astype(np.float16))[:, 7:7 + 256]
    codes, s = od.pack_w4g(host(W.float()), 64)
    wt, sd = bd.pack_weights_w4g(W, 64)
    assert np.array_equal(host(sd), s) and np.array_equal(host(wt), od.w4g_operand(codes))


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (8, 8)])
def test_unaligned_rows_and_padding_untouched(dtype, offset, pad):
    import torch
    M, K, N, group = 5, 288, 21, 32
    _, X, codes, s = make(M, K, N, group, dtype, seed=9)
    buf = torch.full((M, offset + K + pad), float("nan"), dtype=X.dtype, device="cuda")
    Xs = buf[:, offset:offset + K]
    Xs.copy_(X)
    big = torch.full((M + 2, N + 3), 77.0, dtype=out_dt(dtype), device="cuda")
    bd.gemv_w4g(Xs, dev(od.w4g_operand(codes)), dev(s), Y=big[:M, 1:1 + N])
    check(big[:M, 1:1 + N], X, codes, s, group, dtype)
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[:M, 1:1 + N] = False
    assert bool((big[mask] == 77.0).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_non_finite_rows_stay_in_their_rows(dtype):
    """A NaN or infinity reaches exactly its own row; whole rows are NaN because code 0 times an
    infinity is NaN and code c times it is infinite."""
    import torch
    M, K, N, group = 18, 256, 20, 128
    _, X, codes, s = make(M, K, N, group, dtype, seed=10)
    codes[:, 5] = np.where(np.arange(N) % 2 == 0, 3, 0)
    X[2, 5] = float("inf")
    X[17, 9] = float("nan")
    Y = bd.gemv_w4g(X, dev(od.w4g_operand(codes)), dev(s))
    assert bool(torch.isnan(Y[17]).all())
    even = torch.arange(N, device="cuda") % 2 == 0
    assert bool((Y[2][even] == float("inf")).all()) and bool(torch.isnan(Y[2][~even]).all())
    keep = [m for m in range(M) if m not in (2, 17)]
    check(Y[keep], X[keep], codes, s, group, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_small_and_large_values(dtype):
    """Subnormal activations count; the extreme codes are exact; overflow is an infinity."""
    import torch
    K, N, group = 256, 16, 64
    codes = np.full((N, K), -8, np.int8)
    codes[1::2] = 7
    s = np.full((K // group, N), 0.5, np.float16)
    X = torch.zeros((3, K), dtype=tdt(dtype), device="cuda")
    X[0, :] = 2.0 ** -24   # subnormal in fp16
    X[1, 3] = 1.0
    X[2, :] = 60000.0
    Y = bd.gemv_w4g(X, dev(od.w4g_operand(codes)), dev(s))
    check(Y[:2], X[:2], codes, s, group, dtype)
    if dtype != "bf16":
        assert bool(torch.isinf(Y[2]).all())


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_exact_integers(dtype):
    """Integer activations and a power-of-two scale: every sum is exact, so the output is too."""
    rng = np.random.default_rng(12)
    M, K, N, group = 7, 640, 50, 128
    codes = rng.integers(-8, 8, (N, K)).astype(np.int8)
    X = rng.integers(-3, 4, (M, K)).astype(np.float32)
    s = np.full((K // group, N), 0.25, np.float16)
    Y = bd.gemv_w4g(dev(X).to(tdt(dtype)), dev(od.w4g_operand(codes)), dev(s))
    want = (X.astype(np.float64) @ codes.T.astype(np.float64) * 0.25).astype(np.float16)
    assert np.array_equal(host(Y), want)


def test_residual_in_place_and_empty():
    import torch
    M, K, N, group = 4, 128, 24, 64
    _, X, codes, s = make(M, K, N, group, "fp16", seed=13)
    wt, sd = dev(od.w4g_operand(codes)), dev(s)
    Y = torch.randn((M, N), device="cuda").half()
    r = Y.clone()
    bd.gemv_w4g(X, wt, sd, Y=Y, epilogue=bd.EPI_RESIDUAL, residual=Y)
    check(Y, X, codes, s, group, "fp16", "residual", r)
    assert bd.gemv_w4g(X[:0], wt, sd).shape == (0, N)


def test_side_stream_and_graph_replays():
    import torch
    M, K, N, group = 3, 1024, 200, 128
    _, X, codes, s = make(M, K, N, group, "bf16", seed=14)
    wt, sd = dev(od.w4g_operand(codes)), dev(s)
    want = bd.gemv_w4g(X, wt, sd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bd.gemv_w4g(X, wt, sd)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    Y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.gemv_w4g(X, wt, sd, Y=Y)
    for i in range(3):
        X.copy_(torch.randn_like(X, dtype=torch.float32) * (i + 1))
        graph.replay()
        assert torch.equal(Y, bd.gemv_w4g(X, wt, sd)), i
        torch.cuda.synchronize()


def test_repeats_bit_for_bit():
    import torch
    _, X, codes, s = make(8, 16384, 64, 128, "fp16", seed=15)
    wt, sd = dev(od.w4g_operand(codes)), dev(s)
    first = bd.gemv_w4g(X, wt, sd)
    for _ in range(5):
        assert torch.equal(bd.gemv_w4g(X, wt, sd), first)


def test_more_rows_than_one_launch_holds():
    """Rows past the workgroups of one launch (here 1008 rows for 2^20 channels) continue in the next."""
    import torch
    M, K, N, group = 1030, 32, 1 << 20, 32
    g = torch.Generator(device="cuda").manual_seed(0)
    X = torch.randn((M, K), generator=g, device="cuda").half()
    wt = torch.randint(0, 256, (N // 16 * 1024,), generator=g, dtype=torch.uint8, device="cuda")
    s = torch.rand((1, N), generator=g, device="cuda").half()
    r = torch.randn((M, N), generator=g, device="cuda").half()
    Y = bd.gemv_w4g(X, wt, s, epilogue=bd.EPI_RESIDUAL, residual=r)
    for a, b in ((0, 16), (992, 1008), (1008, 1024), (1024, 1030)):
        assert torch.equal(Y[a:b], bd.gemv_w4g(X[a:b], wt, s, epilogue=bd.EPI_RESIDUAL, residual=r[a:b])), a
