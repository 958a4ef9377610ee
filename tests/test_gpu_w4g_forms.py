"""The forms that the group-scaled linear takes for few and many rows, narrow and wide outputs and long sums,
each with several rounds of loads per wave, whole and partial last stages and channels past the last tile.

Integer activations, codes and power-of-two scales keep every partial sum exact in fp32 in any order: |x| <= 3,
|c| <= 8, K <= 16384 and scales 2^-6 or 2^-8 give at most 393216 * 4 units of 2^-8, below 2^24. What is expected
is then the exact sum (formed in fp64) rounded once, equal bit for bit, and one lost k shows. Values that are
not exact are compared with the tolerance of the linear's parity tests."""
import numpy as np
import pytest

from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import host
from test_gpu_w4g import HALF_STEP, out_dt, tdt

pytestmark = pytest.mark.gpu


def weights(N, K, group, seed):
    """(operand, codes fp64 [N, K], scales fp16 [K / group, N]) on the device."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda").to(torch.uint8)
    codes = torch.stack((packed & 15, packed >> 4), -1).view(N, K)
    codes = (codes ^ 8).double() - 8
    s = 2.0 ** torch.randint(-4, -2, (K // group, N), generator=g, device="cuda").mul(2).double()
    return bd.codes_to_w4g(packed, K), codes, s.half()


def dense(codes, s):
    return codes * s.double().t().repeat_interleave(codes.shape[1] // s.shape[0], dim=1)


# (M, K, N): what they reach, for groups 128 and 256; smaller groups take at most the same tiles per workgroup
FORMS = [
    (1, 16384, 50), (4, 8352, 900),                 # four stages per product
    (5, 16384, 50), (8, 10400, 2000),               # two stages per product
    (3, 16384, 2100), (1, 8320, 9000), (4, 4256, 16400),    # one quad of rows: one, two and four tiles
    (8, 4256, 2100), (17, 16384, 50),               # all rows of a product, one tile
    (17, 4256, 4099), (50, 2208, 4099), (33, 2208, 8200),   # two and four tiles, several blocks of rows
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M,K,N", FORMS)
def test_exact_sums(M, K, N, group, dtype):
    import torch
    K = -(-K // group) * group
    K = min(K, 16384)
    wt, codes, s = weights(N, K, group, seed=M + N)
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(tdt(dtype))
    r = torch.randint(-64, 65, (M, N), generator=g, device="cuda").to(out_dt(dtype))
    want = X.double() @ dense(codes, s).t()
    # fp64 holds the sums exactly and so does fp32: the only rounding is the one to the output's type
    assert torch.equal(want.float().double(), want)
    for epi, add in ((bd.EPI_NONE, 0), (bd.EPI_RESIDUAL, r.double())):
        Y = bd.gemv_w4g(X, wt, s, epilogue=epi, residual=r if epi else None)
        exact = (want + add).float()
        assert torch.equal(exact.double(), want + add)
        assert torch.equal(Y, exact.to(out_dt(dtype))), (Y != exact.to(out_dt(dtype))).nonzero()[:5].tolist()


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,K,N,group", [(1, 2080, 16400, 32), (3, 2112, 9000, 64), (2, 2304, 2100, 256),
                                         (17, 1088, 4099, 64), (50, 1056, 8200, 32), (50, 1152, 4099, 128)])
def test_gelu_of_wide_outputs(M, K, N, group, dtype):
    """Normal activations and scales, the tolerance derived in test_gpu_w4g: (parts K + 3 groups + 32) 2^-23 of
    sum |x||c|s, times GELU's largest slope, 2^-15 of the result for GELU itself, and the output's half step."""
    import torch
    wt, codes, s = weights(N, K, group, seed=N)
    g = torch.Generator(device="cuda").manual_seed(K)
    s = (s.float() * (0.5 + torch.rand(s.shape, generator=g, device="cuda"))).half()
    X = torch.randn((M, K), generator=g, device="cuda").to(tdt(dtype))
    W = dense(codes, s)
    y, size = X.double() @ W.t(), X.double().abs() @ W.abs().t()
    y = y * torch.special.ndtr(y)
    parts = 3 if dtype == "fp32" else 1
    t = 1.13 * (parts * K + 3 * (K // group) + 32) * 2.0 ** -23 * size + 2.0 ** -15 * y.abs()
    t = t + HALF_STEP[dtype] * (y.abs() + t) + 2.0 ** -25
    err = (bd.gemv_w4g(X, wt, s, epilogue=bd.EPI_GELU).double() - y).abs()
    assert bool((err <= t).all()), float((err / t).max())


@pytest.mark.parametrize("M,N", [(2, 40), (7, 1500), (4, 2100), (12, 100), (30, 4200), (3, 16400)])
def test_every_part_of_an_fp32_activation_counts(M, N):
    """Two activations that cancel but for their last bits, on equal codes: what is left is a part of the
    activation that 16 bits do not hold. All sums are exact, so the result is."""
    import torch
    K, group = 416, 32
    wt, codes, s = weights(N, K, group, seed=N)
    s = torch.full_like(s, 2.0 ** 10)
    pairs = np.random.default_rng(M).choice(K, (M, 2), replace=False).tolist()
    X = torch.zeros((M, K), device="cuda")
    for m, (k1, k2) in enumerate(pairs):
        left = (2.0 ** -10, 3 * 2.0 ** -18, 2.0 ** -20)[m % 3]
        X[m, k1] = 1 + 2.0 ** -9 + left
        X[m, k2] = -(1 + 2.0 ** -9)
        codes[:, k2] = codes[:, k1]
        assert float(X[m, k1]) == 1 + 2.0 ** -9 + left
    u = (codes.long() & 15).to(torch.uint8)
    packed = (u[:, 0::2] | (u[:, 1::2] << 4)).contiguous()
    want = X.double() @ dense(codes, s).t()
    Y = bd.gemv_w4g(X, bd.codes_to_w4g(packed, K), s)
    assert torch.equal(Y, want.float().half())
    assert np.count_nonzero(host(Y)) > 0.8 * Y.numel()
