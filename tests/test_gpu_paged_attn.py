"""GPU parity of the one-token attention over the paged cache against the fp64 oracle.

Tolerance per (sequence, head, channel) from the arithmetic. A score is a sum of D fp32 terms: off by
at most (D + 4) 2^-23 |scale| sum |q||k|, and its product with log2 e and the difference to the
maximum by 3 * 2^-23 |s| each; exp2 adds 2^-22. That is the relative error d of a weight p, for the
largest |q||k| among the visible keys. The two 16-bit parts of p leave 2^-17 of it, and sums over n
keys (n + 64) 2^-23. Numerator and denominator each carry these, relative to A = sum p|v| / sum p, so
|error| <= A (2 d + 2^-17 + 2 (n + 64) 2^-23), to which the output's half step is added."""
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


class Batch:
    """A batch over a cache whose unused slots, unused table entries and spare pages are all NaN / bad."""

    def __init__(self, lens, H, KV, D, page, dtype, seed=0, qscale=1.5, spare=3):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.KV, self.D, self.page, self.dtype = list(lens), H, KV, D, page, dtype
        B = len(lens)
        used = [-(-max(n, 0) // page) for n in lens]
        self.P = sum(used) + spare
        self.kc = torch.full((self.P, KV, page, D), float("nan"), dtype=tdt(dtype), device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        ids = rng.permutation(self.P)
        table = np.full((B, max(used + [1]) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(lens):
            table[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
            for i in range(used[b]):
                m = min(page, n - i * page)
                for c in (self.kc, self.vc):
                    c[int(table[b, i]), :, :m] = dev(rng.standard_normal((KV, m, D)).astype(np.float32)).to(c.dtype)
        self.table = dev(table)
        self.q = dev((qscale * rng.standard_normal((B, H, D))).astype(np.float32)).to(tdt(dtype))
        self.ld = dev(np.array(lens, np.int32))

    def run(self, **kw):
        return bd.paged_attn_decode(self.q, self.kc, self.vc, self.table, self.ld, **kw)

    def check(self, out, scale=None, window=0, sinks=0, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        q, kc, vc, table = f64(self.q), f64(self.kc), f64(self.vc), host(self.table)
        got = f64(out)
        want = od.paged_attention(q, kc, vc, table, self.lens, scale, window, sinks)
        for b in range(len(self.lens)) if rows is None else rows:
            j = od.visible(self.lens[b], window, sinks)
            if not j.size or np.isnan(want[b]).any():
                assert np.array_equal(got[b], want[b], equal_nan=True), b
                continue
            ids, off = table[b, j // self.page], j % self.page
            for h in range(self.H):
                k, v = kc[ids, h * self.KV // self.H, off], vc[ids, h * self.KV // self.H, off]
                s = k @ q[b, h] * scale
                p = np.exp(s - s.max())
                size = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
                d = ((self.D + 4) + 6) * 2.0 ** -23 * size * 2 + 2.0 ** -22
                A = (p / p.sum()) @ np.abs(v)
                tol = A * (2 * d + 2.0 ** -17 + 2 * (j.size + 64) * 2.0 ** -23)
                tol = tol + HALF_STEP[self.dtype] * (np.abs(want[b, h]) + tol) + 2.0 ** -25
                err = np.abs(got[b, h] - want[b, h])
                assert np.all(err <= tol), (b, h, float((err / tol).max()))


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 257]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,KV,D,page", [(1, 1, 64, 16), (8, 1, 256, 16), (6, 2, 96, 32), (4, 4, 128, 64),
                                         (16, 1, 192, 16), (10, 2, 64, 128), (17, 1, 128, 16),
                                         (40, 2, 64, 16)])
def test_lengths(H, KV, D, page, dtype):
    b = Batch(EDGES, H, KV, D, page, dtype, seed=H + D)
    b.check(b.run())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [1, 700, 1001, 5000])
def test_one_sequence_split_and_joined(n, dtype):
    b = Batch([n], 8, 2, 128, 16, dtype, seed=n)
    out = b.run()
    b.check(out)
    import torch
    for limit in (n, 1, 40, 4 * n):   # how the work is split does not have to match the length
        b.check(b.run(max_len=limit))
    assert torch.equal(out, b.run())


WINDOWS = [(1, 0), (1, 1), (5, 0), (16, 4), (32, 0), (33, 1), (100, 4), (100, 40), (64, 64), (1000, 3), (31, 33)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_and_sinks(window, sinks, dtype):
    b = Batch(EDGES + [600, 1031], 4, 2, 64, 16, dtype, seed=window)
    b.check(b.run(window=window, sinks=sinks), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("KV,D", [(2, 64), (16, 96), (1, 256)])
def test_one_workgroup_per_row(KV, D, dtype):
    """Rows enough for one workgroup each up to 32 tiles, and a max_len that is shorter than the sequences."""
    rng = np.random.default_rng(D)
    b = Batch([0, 1024, 1, 255, 1009] + list(rng.integers(0, 700, 11)), KV, KV, D, 32, dtype, seed=D)
    for max_len in (1024, 256, 1, 0):
        b.check(b.run(max_len=max_len))
    b.check(b.run(max_len=200, window=700, sinks=40), window=700, sinks=40)


def test_window_reads_no_hidden_page():
    """Pages without a visible token may be gone from the table and hold anything."""
    import torch
    b = Batch([500, 333, 64], 4, 1, 64, 16, "fp16", seed=2)
    window, sinks = 70, 20
    want = b.run(window=window, sinks=sinks)
    for i, n in enumerate(b.lens):
        seen = set((od.visible(n, window, sinks) // 16).tolist())
        for p in range(b.table.shape[1]):
            if p not in seen:
                b.table[i, p] = -7 if p % 2 else 1 << 30
    got = b.run(window=window, sinks=sinks)
    assert torch.equal(got, want)
    b.check(got, window=window, sinks=sinks)


@pytest.mark.parametrize("entry", [-1, -(1 << 31), 1 << 20, (1 << 31) - 1])
def test_bad_page_poisons_its_sequence_only(entry):
    import torch
    b = Batch([300, 300, 300, 40], 4, 2, 64, 16, "bf16", seed=3)
    b.table[1, 7] = entry
    b.table[3, 2] = b.P           # one past the last page, holding the last tokens
    for kw in ({}, dict(max_len=1)):
        out = b.run(**kw)
        assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3]).all())
        b.check(out, rows=[0, 2])


def test_length_beyond_the_table_and_negative():
    import torch
    b = Batch([100, 100, 100, 100], 2, 1, 64, 16, "fp16", seed=4)
    b.ld[1] = b.table.shape[1] * 16 + 1
    b.ld[2] = -5
    b.ld[3] = (1 << 31) - 1
    out = b.run()
    assert bool(torch.isnan(out[1]).all()) and bool((out[2] == 0).all()) and bool(torch.isnan(out[3]).all())
    b.check(out, rows=[0])
    out = b.run(window=10, sinks=2)
    assert bool(torch.isnan(out[1]).all()) and bool((out[2] == 0).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_peaked_and_flat_weights(dtype):
    """One key that outweighs all others, all keys alike, reversed and large scales."""
    b = Batch([1500, 77], 4, 1, 128, 16, dtype, seed=5, qscale=8.0)
    for scale in (1.0, 0.0, -0.3, 0.001):
        b.check(b.run(scale=scale), scale=scale)


def test_small_weights_add_up():
    """Thousands of keys whose weight is below fp16's smallest number still count together."""
    import torch
    n = 40000
    b = Batch([n], 1, 1, 64, 64, "fp16", seed=6)
    b.kc[:] = 0
    b.vc[:] = 1.0
    b.q[:] = 0
    b.q[0, 0, 0] = 1.0
    b.kc[int(b.table[0, 0]), 0, 0, 0] = 17.5
    b.vc[int(b.table[0, 0]), 0, 0] = 0.0
    rest = (n - 1) * np.exp(-17.5)
    got = b.run(scale=1.0)
    want = rest / (1 + rest)
    assert np.all(np.abs(f64(got) - want) <= want * (2.0 ** -11 + 2.0 ** -12))
    assert torch.isfinite(got).all()


def test_infinite_and_nan_keys():
    """A visible infinity in a key's channel makes its heads NaN as the formula does; others stay."""
    import torch
    b = Batch([90, 90], 4, 2, 64, 16, "fp16", seed=7)
    b.kc[int(b.table[0, 1]), 0, 3, 5] = float("inf")
    b.vc[int(b.table[0, 2]), 1, 2, 9] = float("nan")
    b.q[0, 0, 5] = 1.0
    b.q[0, 1, 5] = -1.0        # score -inf: the key simply does not count
    out = b.run()
    assert bool(torch.isnan(out[0, 0]).all())
    assert bool(torch.isfinite(out[0, 1]).all())
    assert bool(torch.isnan(out[0, 2:, 9]).all())
    ok = torch.arange(64, device="cuda") != 9
    assert bool(torch.isfinite(out[0, 2:][:, ok]).all())
    b.check(out, rows=[1])


def test_every_score_minus_infinity():
    """Softmax of nothing but -inf is NaN (0 / 0), unlike a sequence without visible tokens."""
    import torch
    b = Batch([700], 2, 2, 64, 16, "bf16", seed=8)
    b.kc[:, 0, :, 0] = float("-inf")
    b.q[:, 0, 0] = 1.0
    out = b.run()
    assert bool(torch.isnan(out[0, 0]).all()) and bool(torch.isfinite(out[0, 1]).all())


@pytest.mark.parametrize("offset", [0, 1, 8])
def test_strides_and_padding_untouched(offset):
    """q a slice of a wider row, out a slice of a padded buffer, keys and values of a page side by side."""
    import torch
    H, KV, D, page = 6, 3, 64, 16
    b = Batch([100, 0, 40], H, KV, D, page, "fp16", seed=9)
    want = b.run()
    wide = torch.full((3, offset + H * D + 5), float("nan"), dtype=b.q.dtype, device="cuda")
    q = wide[:, offset:offset + H * D].unflatten(1, (H, D))
    q.copy_(b.q)
    both = torch.full((b.P, 2, KV, page, D), float("nan"), dtype=b.q.dtype, device="cuda")
    both[:, 0], both[:, 1] = b.kc, b.vc
    big = torch.full((5, offset + H * D + 3), 9.0, dtype=b.q.dtype, device="cuda")
    out = big[:3, offset:offset + H * D].unflatten(1, (H, D))
    bd.paged_attn_decode(q, both[:, 0], both[:, 1], b.table, b.ld, out=out)
    assert torch.equal(out, want)
    big[:3, offset:offset + H * D] = 9.0
    assert bool((big == 9.0).all())


def test_cache_past_32_bits():
    import torch
    KV, D, page = 8, 128, 256
    P = (1 << 31) // (KV * D * page) + 2
    kc = torch.empty((P, KV, page, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    b = Batch([500, 300], 16, KV, D, page, "bf16", seed=10)
    small = b.run()
    far = torch.tensor([P - 1, P - 2, P // 2 + 5, 1], device="cuda")
    table = b.table.clone()
    at = 0
    for i, n in enumerate(b.lens):
        for p in range(-(-n // page)):
            src, dst = int(table[i, p]), int(far[at])
            kc[dst], vc[dst] = b.kc[src], b.vc[src]
            table[i, p] = dst
            at += 1
    assert torch.equal(bd.paged_attn_decode(b.q, kc, vc, table, b.ld), small)


def test_graph_replays_with_growing_lengths():
    """One captured graph serves growing sequences; two graphs with workspaces of their own and eager calls
    between them do not disturb each other."""
    import torch
    b = Batch([400, 900, 17], 8, 2, 128, 16, "bf16", seed=11)
    full = list(b.lens)
    outs = [torch.empty_like(b.q) for _ in range(2)]
    b.run()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(out=o)
        graphs.append(g)
    for cut in (0, 1, 16, 390):
        b.lens = [max(n - cut, 0) for n in full]
        b.ld.copy_(torch.tensor(b.lens, dtype=torch.int32))
        graphs[0].replay()
        graphs[1].replay()
        eager = b.run()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager), cut
        b.check(eager)
        torch.cuda.synchronize()


@pytest.mark.parametrize("n", [2000, 20000])
def test_side_stream_and_caller_workspace(n):
    import torch
    b = Batch([n], 4, 1, 64, 16, "fp16", seed=12)
    want = b.run()
    need = bd.lib().w4a4_paged_attn_workspace_bytes(1, 4, 1, 64, b.table.shape[1] * 16, 0, 0)
    assert need > 0 or n == 2000            # the longer one is split and joined
    # NaN bytes: nothing stale is read
    ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(b.run(ws=ws), want)
    if need:
        with pytest.raises(bd.W4A4Error, match="workspace"):
            b.run(ws=ws[:need - 256])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_empty_batch():
    b = Batch([5, 6], 2, 1, 64, 16, "fp16")
    out = bd.paged_attn_decode(b.q[:0], b.kc, b.vc, b.table[:0], b.ld[:0])
    assert out.shape == (0, 2, 64)
