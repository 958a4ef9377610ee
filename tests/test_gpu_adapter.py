"""GPU parity of the low-rank adapters against the fp64 oracle.

Tolerance per output from the arithmetic. An inner product of K exact products, summed in fp32 in any order and joined
from up to 64 parts, is off by (K + 64) 2^-23 sum |x||a|; the two 16-bit parts leave 2^-17 of it (bf16; fp16 less, and
2^-24 of its 32 ranks' largest); the outer sum of R terms adds (R + 8) 2^-23 sum |b||t|. Times |scale| (rounded once),
added to Y in fp32 (2^-23 of the result), and rounded once to 16 bits. GELU has slope at most 1.13 and its own evaluation
is within 2^-15 relative."""
import numpy as np
import pytest

from oracle import served as osv
from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import dev
from test_gpu_norm_rope import f64, tdt

pytestmark = pytest.mark.gpu
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
EPIS = {"none": bd.EPI_NONE, "gelu": bd.EPI_GELU, "residual": bd.EPI_RESIDUAL}


class Case:
    def __init__(self, M, K, N, R, n, dtype, seed=0, ids=None, xscale=1.0):
        rng = np.random.default_rng(seed)
        t = lambda *s: dev(rng.standard_normal(s).astype(np.float32)).to(tdt(dtype))  # noqa: E731
        self.dtype = dtype
        self.X, self.Y, self.res = t(M, K) * xscale, t(M, N), t(M, N)
        self.A, self.B = t(n, R, K) * K ** -0.5, t(n, N, R) * 0.2
        self.scale = dev((0.5 + rng.random(n)).astype(np.float32))
        self.ids = dev((rng.integers(-1, n, M) if ids is None else np.asarray(ids)).astype(np.int32))

    def run(self, epi="none", **kw):
        a = dict(Y=self.Y, X=self.X, A=self.A, B=self.B, ids=self.ids, scale=self.scale, epilogue=EPIS[epi],
                 residual=self.res if epi == "residual" else None) | kw
        return bd.adapter_add(**a)

    def check(self, out, epi="none", scale=True, rows=None):
        K, R = self.A.shape[2], self.A.shape[1]
        with np.errstate(invalid="ignore"):
            y, inner, outer, pre = osv.adapter_add(
                *(f64(t) for t in (self.Y, self.X, self.A, self.B)), self.ids.tolist(),
                f64(self.scale) if scale else None, epi, f64(self.res))
        tol = (K + 64) * 2.0 ** -23 * inner + (2.0 ** -17 + (R + 8) * 2.0 ** -23 + 2.0 ** -23) * outer
        tol = tol + 2.0 ** -23 * np.abs(pre)
        if epi == "gelu":
            tol = 1.13 * tol + 2.0 ** -15 * np.abs(y)
        elif epi == "residual":
            tol = tol + 2.0 ** -23 * np.abs(y)
        tol = tol + HALF_STEP[self.dtype] * (np.abs(y) + tol) + 2.0 ** -25
        got, fine = f64(out), np.isfinite(y)      # an oracle that is not finite wants the same infinity or a NaN
        assert np.array_equal(got[~fine], y[~fine], equal_nan=True)
        err, tol = np.where(fine, np.abs(got - y), 0.0), np.where(fine, tol, 0.0)
        if rows is not None:
            err, tol = err[rows], tol[rows]
        assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:5])


CASES = [(1, 8, 1, 8, 1), (1, 1024, 1000, 16, 3), (2, 24, 5, 24, 2), (7, 520, 63, 8, 9), (15, 256, 64, 16, 4),
         (16, 264, 65, 40, 20), (17, 2048, 130, 32, 5), (33, 96, 257, 64, 1), (50, 1024, 515, 16, 50),
         (100, 336, 100, 128, 7), (300, 160, 33, 72, 3), (5, 4096, 48, 256, 3), (2200, 64, 40, 16, 6)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N,R,n", CASES)
def test_adapters(M, K, N, R, n, dtype):
    c = Case(M, K, N, R, n, dtype, seed=M + K)
    for epi in ("none", "gelu", "residual") if M < 300 else ("none",):
        c.check(c.run(epi), epi)
    c.check(c.run(scale=None), scale=False)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("ids", [[-1] * 20, [0] * 20, [3] * 10 + [1] * 10, list(range(16)) + [2, 2, -1, 40],
                                 [5, -(1 << 31), (1 << 31) - 1, 16, 15] * 4])
def test_which_adapter(ids, dtype):
    """One for all, one each, none at all, ids that name no adapter."""
    import torch
    c = Case(20, 128, 100, 16, 16, dtype, seed=1, ids=ids)
    for epi in EPIS:
        c.check(c.run(epi), epi)
    none = [m for m, i in enumerate(ids) if not 0 <= i < 16]
    assert torch.equal(c.run()[none], c.Y[none])


@pytest.mark.parametrize("epi", list(EPIS))
def test_in_place(epi):
    import torch
    c = Case(37, 256, 333, 24, 4, "bf16", seed=2)
    want = c.run(epi)
    y = c.Y.clone()
    assert c.run(epi, Y=y, out=y) is not None and torch.equal(y, want)
    y = c.Y.clone()
    c.run(epi, Y=y, out=y)                     # again from the same state
    assert torch.equal(y, want)
    if epi == "residual":
        r = c.res.clone()
        c.run(epi, residual=r, out=r)
        assert torch.equal(r, want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_touch_each_other(bad):
    """An adapter, or a row, that is not finite is its own rows' matter."""
    import torch
    c = Case(40, 256, 100, 16, 3, "fp16", seed=3, ids=[0, 1, 2, -1] * 10)
    want = c.run()
    c.A[1, 5, 7] = bad
    c.B[1, 9, 3] = bad
    c.X[2, 0] = bad
    out = c.run()
    hurt = torch.zeros(40, dtype=torch.bool, device="cuda")
    hurt[1::4] = True
    hurt[2] = True
    assert torch.equal(out[~hurt], want[~hurt])
    assert not bool(torch.isfinite(out[hurt]).all(1).any())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("xscale", [30000.0, 8000.0, 2.0 ** -20])
def test_inner_products_outside_fp16(xscale, dtype):
    """Inner products far above 65504 and far below fp16's smallest number keep their bits (30000 takes some elements
    of X beyond fp16 themselves: those rows are infinite or NaN)."""
    c = Case(9, 512, 70, 16, 2, dtype, seed=4, xscale=xscale)
    c.A, c.B = c.A * (40.0 if xscale > 1 else 1.0), c.B * (2.0 ** -20 if xscale > 1 else 8.0)
    c.Y = c.Y * 0
    c.check(c.run())


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strides_and_padding_untouched(offset):
    import torch
    M, K, N, R, n = 21, 136, 77, 16, 3
    c = Case(M, K, N, R, n, "fp16", seed=5)
    want = c.run("residual")

    def wide(t, extra=6):
        big = torch.full((t.shape[0], offset + t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
        view = big[:, offset:offset + t.shape[1]]
        view.copy_(t)
        return view
    both = torch.full((n, R * K + N * R + 3), float("nan"), dtype=c.A.dtype, device="cuda")
    A = both[:, 1:1 + R * K].unflatten(1, (R, K))
    B = both[:, 2 + R * K:2 + R * K + N * R].unflatten(1, (N, R))
    A.copy_(c.A), B.copy_(c.B)
    big = torch.full((M + 2, offset + N + 5), 9.0, dtype=c.Y.dtype, device="cuda")
    out = big[:M, offset:offset + N]
    c.run("residual", Y=wide(c.Y), X=wide(c.X), A=A, B=B, residual=wide(c.res), out=out)
    assert torch.equal(out, want)
    out.fill_(9.0)
    assert bool((big == 9.0).all())


def test_graph_follows_the_ids():
    import torch
    c = Case(50, 512, 200, 32, 6, "bf16", seed=6)
    out = torch.empty_like(c.Y)
    c.run("gelu", out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run("gelu", out=out)
    for turn in range(4):
        c.ids.copy_(torch.randint(-1, 6, (50,), dtype=torch.int32))
        out.zero_()
        g.replay()
        got = out.clone()
        eager = c.run("gelu")
        assert torch.equal(got, eager), turn
        c.check(eager, "gelu")
        torch.cuda.synchronize()


def test_side_stream_workspace_and_empty():
    import torch
    c = Case(30, 2048, 100, 16, 4, "fp16", seed=7)
    want = c.run()
    need = bd.lib().w4a4_adapter_workspace_bytes(30, 2048, 16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(ws=ws), want)
    with pytest.raises(bd.W4A4Error, match="workspace"):
        c.run(ws=ws[:need - 256])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    none = bd.adapter_add(c.Y[:0], c.X[:0], c.A, c.B, c.ids[:0], c.scale)
    assert none.shape == (0, 100)


def test_same_bits_whatever_is_beside_a_row():
    """A row's result does not depend on the other rows of its tile, nor on how often it is asked for."""
    import torch
    c = Case(16, 256, 90, 24, 5, "fp16", seed=8)
    out = c.run()
    assert torch.equal(out, c.run())
    c.ids[1::2] = -1
    again = c.run()
    assert torch.equal(again[0::2], out[0::2])
