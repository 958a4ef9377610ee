"""Edges of the serving calls that sizes and arguments allow. Oracle and tolerances as in the tests of each call."""
import numpy as np
import pytest

from oracle import served as osv
from w4a4_post_quantized_zigzag_amd import binding as bd
from w4a4_post_quantized_zigzag_amd.stack import Attention, PagedCache

from test_gpu_adapter import EPIS, HALF_STEP, Case
from test_gpu_kv_attn import Batch
from test_gpu_norm_rope import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["fp16", "int8", "fp4"])
def test_slots_outside_every_kind_of_cache(kind):
    """Whatever a cache holds, a slot outside it is skipped, reads as zeros and touches nothing."""
    import torch
    A = Attention(4, 2, 64)
    cache, want = [PagedCache(1, A, 1, pages=4, kv=kind) for _ in range(2)]
    k, v = (torch.randn(6, 2, 64, device="cuda").half() for _ in range(2))
    at = torch.tensor([-1, 64, 63, 1 << 40, -(1 << 40), 0], device="cuda")
    cache.write(0, k, v, at)
    want.write(0, k[[2, 5]], v[[2, 5]], at[[2, 5]])
    assert all(torch.equal(a, b) for a, b in zip(cache.kv[0], want.kv[0]))
    for got, kept in zip(cache.read(0, at), want.read(0, at[[2, 5]])):
        assert torch.equal(got[[2, 5]], kept) and bool(kept.any()) and not bool(got[[0, 1, 3, 4]].any())


@pytest.mark.parametrize("kind", ["none", "int8", "fp4"])
@pytest.mark.parametrize("B,H,KV,D", [(513, 8, 1, 64), (300, 32, 2, 128), (2060, 4, 1, 64)])
def test_prefix_for_more_rows_than_an_xcd_has_workgroups(B, H, KV, D, kind):
    """More than 4096 query rows a key/value head: runs of row blocks, the last one not full."""
    lens = [(5 * b) % 37 for b in range(B)]
    b = Batch(lens, H, KV, D, 16, "fp16" if B == 513 else "bf16", kind, prefix=1003, seed=B)
    b.check(b.run(max_len=36), rows=[0, 1, 127, 255, B // 2, B - 2, B - 1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("R", [16, 64])
@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("up,down", [(2.0 ** 14, 2.0 ** -8), (2.0 ** 16, 2.0 ** -14)])
def test_a_rank_far_above_the_others(up, down, M, R, dtype):
    """A rank 2^22 or 2^30 above the others that no channel takes anything from. In fp16 the second part of an inner product
    that is far below the largest of its 32 is a subnormal number: at the scale that takes the largest to 2^14 or above its
    half step is 2^-25, 2^-39 of the largest."""
    c = Case(M, 256, 90, R, 3, dtype, seed=R)
    c.A *= down
    c.A[:, 3] *= up / down
    c.B *= 1 / down
    c.B[:, :, 3] = 0
    c.Y *= 0
    assert bool(c.A.isfinite().all()) and bool(c.B.isfinite().all())
    X, A, B, ids, scale = f64(c.X), f64(c.A), f64(c.B), c.ids.tolist(), f64(c.scale)
    y, inner, outer, _ = osv.adapter_add(f64(c.Y), X, A, B, ids, scale, "none", None)
    tol = (256 + 64) * 2.0 ** -23 * inner + (2.0 ** -17 + (R + 9) * 2.0 ** -23) * outer
    if dtype == "fp16":
        for m, i in enumerate(ids):
            for g in range(0, R if i >= 0 else 0, 32):
                top = np.abs(A[i, g:g + 32] @ X[m]).max() * (1 + 2.0 ** -10)
                tol[m] += 2.0 ** -39 * top * scale[i] * np.abs(B[i, :, g:g + 32]).sum(1)
    tol = tol + 2.0 ** -23 * np.abs(y)
    tol = tol + HALF_STEP[dtype] * (np.abs(y) + tol) + 2.0 ** -25
    err = np.abs(f64(c.run()) - y)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("kind", ["int8", "fp4"])
@pytest.mark.parametrize("M", [4, 700])
def test_two_rows_with_one_slot(M, kind):
    """Every code and scale there is one of the two rows', every other slot as without them."""
    import torch
    KV, D, page, pages = 2, 128, 16, 50
    k, v = (torch.randn(M, KV, D, device="cuda").half() * s for s in (1.0, 40.0))
    q = torch.randn(M, 4, D, device="cuda").half()
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(M))[:M].cuda()
    for append in (lambda c, at: bd.kv_append_quant(k, v, c, at),
                   lambda c, at: bd.qk_norm_rope_append_quant(q, k, v, None, None, None, None, c, at)):
        caches = [bd.quant_pages(pages, KV, page, D, kind) for _ in range(3)]
        twice, first, second = slots.clone(), slots.clone(), slots.clone()
        twice[1] = slots[M - 1]
        first[1], first[M - 1] = slots[M - 1], -1
        second[1] = -1
        for cache, at in zip(caches, (twice, first, second)):
            append(cache, at)
        for got, a, b in zip(*caches):
            assert bool(((got.view(torch.uint8) == a.view(torch.uint8)) | (got.view(torch.uint8) == b.view(torch.uint8))).all())


@pytest.mark.parametrize("epi", list(EPIS))
@pytest.mark.parametrize("M,N,R,n", [(300, 333, 24, 4), (700, 1030, 64, 20), (1030, 77, 16, 3)])
def test_in_place_over_many_rows(M, N, R, n, epi):
    """More than 256 rows, as the stack calls it: the next block's Y is on its way while this one is stored, and rows
    without an adapter are left alone."""
    import torch
    c = Case(M, 264, N, R, n, "bf16", seed=M)
    assert -1 in c.ids.tolist()
    want = c.run(epi)
    c.check(want, epi)
    y = torch.full((M + 1, N + 3), 7.0, dtype=c.Y.dtype, device="cuda")
    out = y[:M, 2:2 + N]
    for _ in range(3):
        out.copy_(c.Y)
        c.run(epi, Y=out, out=out)
        assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((y == 7.0).all())
    if epi == "residual":
        r = c.res.clone()
        c.run(epi, residual=r, out=r)
        assert torch.equal(r, want)


@pytest.mark.parametrize("M,R", [(500, 8), (65, 16)])
def test_adapters_in_several_launches(M, R):
    """2^22 channels and more take several launches of some tiles of rows each: the same bits as on slices of the channels,
    whose calls are one launch."""
    import torch
    N, K, n, part = (1 << 22) + 13 if M > 256 else (1 << 24) - 3, 40, 2, 4096
    t = lambda *s: torch.randn(*s, dtype=torch.bfloat16, device="cuda", generator=g)  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(M)
    X, A, B, Y = t(M, K), t(n, R, K), t(n, N, R), t(M, N)
    ids = torch.randint(-1, n, (M,), dtype=torch.int32, device="cuda", generator=g)
    out = bd.adapter_add(Y, X, A, B, ids)
    for at in (0, 1 << 20, N // 2 + 1, N - part):
        want = bd.adapter_add(Y[:, at:at + part].contiguous(), X, A, B[:, at:at + part].contiguous(), ids)
        assert torch.equal(out[:, at:at + part], want), at
    for rows in (slice(0, 64), slice(M - 64, M)):
        none = ids[rows] < 0
        assert torch.equal(out[rows][none], Y[rows][none]) and not torch.equal(out[rows][~none], Y[rows][~none])


@pytest.mark.parametrize("kind", ["none", "int8", "fp4"])
@pytest.mark.parametrize("power", [88, -40])
def test_values_far_from_one(power, kind):
    """bf16 values up to 2^88 and far below one, behind scores that grow from tile to tile: a power of two on all values is
    that power on the results, bit for bit."""
    import torch
    b = Batch([900, 33, 0, 2500], 8, 2, 128, 16, "bf16", kind, prefix=777, seed=9, qscale=6.0)
    calls = [b.shared] + ([lambda: bd.paged_attn_decode_quant(b.q, b.cache, b.table, b.ld)] if kind != "none" else [])
    want = [f() for f in calls]
    b.check(want[0])
    shift = power - int(np.ceil(np.log2(np.nanmax(np.abs(b.values[1])))))
    if kind == "fp4":
        b.cache[3].add_((b.cache[3] != 255).to(torch.uint8) * (shift % 256))
    else:
        b.cache[1 if kind == "none" else 3].mul_(2.0 ** shift)
    for f, w in zip(calls, want):
        got = f()
        assert bool(got.isfinite().all()) and torch.equal(got.double(), w.double() * 2.0 ** shift)
