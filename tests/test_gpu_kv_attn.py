"""GPU parity of the one-token attention over a quantized cache, and behind a shared prefix, against the fp64 oracle.

Tolerance as for the 16-bit cache (test_gpu_paged_attn.py), which holds here with two more fp32 roundings: a score is a
sum of D exact products, off by at most (D + 4) 2^-23 |scale| sum |q||k|, times the key's scale, the call's scale and
log2 e and less the maximum, 5 * 2^-23 |s|; exp2 adds 2^-22: the relative error d of a weight. The value's scale rounds
the weight once more (2^-24), the two 16-bit parts leave 2^-17 of it, and sums over n keys, joined from up to 256 parts,
(n + 320) 2^-23. With A = sum p|v| / sum p, |error| <= A (2 d + 2^-17 + 2 (n + 320) 2^-23), to which the output's half
step is added."""
import numpy as np
import pytest

from oracle import decode as od
from oracle import served as osv
from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import dev, host
from test_gpu_norm_rope import f64, tdt

pytestmark = pytest.mark.gpu
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
KINDS = ["int8", "fp4"]


class Batch:
    """Sequences (and a prefix) over a cache whose unused slots, unused table entries and spare pages hold the worst:
    NaN scales and any code, NaN elements, page numbers that do not exist."""

    def __init__(self, lens, H, KV, D, page, dtype, kind, prefix=0, seed=0, qscale=1.5, spare=3):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.KV, self.D, self.page, self.dtype, self.kind = list(lens), H, KV, D, page, dtype, kind
        self.prefix = prefix
        pages = lambda n: -(-max(n, 0) // page)  # noqa: E731
        used, front = [pages(n) for n in lens], pages(prefix)
        self.P = P = sum(used) + front + spare
        ids = rng.permutation(P)
        table = np.full((len(lens), max(used + [1]) + 1), -1, np.int32)
        at, live = front, np.zeros((P, page), bool)
        for b, n in enumerate(lens):
            table[b, :used[b]] = ids[at:at + used[b]]
            at += used[b]
            for i in range(used[b]):
                live[table[b, i], :min(page, n - i * page)] = True
        pt = np.concatenate([ids[:front], [-1]]).astype(np.int32)
        for i in range(front):
            live[pt[i], :min(page, prefix - i * page)] = True
        hide = ~live[:, None, :]                       # [P, 1, page]
        self.values, arrays = [], []
        for _ in range(2):
            x = torch.from_numpy(rng.standard_normal((P, KV, page, D)).astype(np.float32)).to(tdt(dtype)).double().numpy()
            if kind == "none":
                x[np.broadcast_to(hide, x.shape[:3])] = np.nan
                self.values.append(x)
                arrays.append((torch.from_numpy(x).to(tdt(dtype)), None))
                continue
            if kind == "int8":
                c, s = osv.quant_int8(x)
                v = osv.values_int8(c, s)
                h = np.broadcast_to(hide, s.shape)
                s = np.where(h, np.float32("nan"), s)
            else:
                c, s = osv.quant_fp4(x, dtype)
                v = osv.values_fp4(c, s)
                h = np.broadcast_to(hide, c.shape[:3])
                c[h] = rng.integers(0, 16, (int(h.sum()), D))
                c, s = osv.pack_fp4(c), np.where(h[..., None], 255, s).astype(np.uint8)
                s = np.ascontiguousarray(s.transpose(0, 1, 3, 2))
            v[np.broadcast_to(hide, v.shape[:3])] = np.nan
            if kind == "int8":
                c[h] = rng.integers(-127, 128, (int(h.sum()), D))
            self.values.append(v)
            arrays.append((torch.from_numpy(np.ascontiguousarray(c)), torch.from_numpy(np.ascontiguousarray(s))))
        cache = [a[0].cuda() for a in arrays] + ([] if kind == "none" else [a[1].cuda() for a in arrays])
        self.cache = tuple(cache)
        self.table, self.pt = dev(table), dev(pt)
        self.q = dev((qscale * rng.standard_normal((len(lens), H, D))).astype(np.float32)).to(tdt(dtype))
        self.ld = dev(np.array(lens, np.int32))
        self.pl = dev(np.array([prefix], np.int32))

    def run(self, **kw):
        if self.kind == "none" or self.prefix or "max_prefix" in kw:
            return bd.paged_attn_shared(self.q, self.cache, self.pt, self.pl, self.table, self.ld, **kw)
        return bd.paged_attn_decode_quant(self.q, self.cache, self.table, self.ld, **kw)

    def shared(self, **kw):
        return bd.paged_attn_shared(self.q, self.cache, self.pt, self.pl, self.table, self.ld, **kw)

    def check(self, out, scale=None, window=0, sinks=0, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        q, table, pt = f64(self.q), host(self.table), host(self.pt)
        kc, vc = self.values
        got = f64(out)
        if window:
            want = od.paged_attention(q, kc, vc, table, self.lens, scale, window, sinks)
        else:
            want = osv.shared_attention(q, kc, vc, pt, self.prefix, table, self.lens, scale)
        jp = np.arange(self.prefix)
        for b in range(len(self.lens)) if rows is None else rows:
            j = od.visible(self.lens[b], window, sinks)
            if not j.size + self.prefix or np.isnan(want[b]).any():
                assert np.array_equal(got[b], want[b], equal_nan=True), b
                continue
            ids = np.concatenate([pt[jp // self.page], table[b, j // self.page]])
            off = np.concatenate([jp % self.page, j % self.page])
            n = ids.size
            for h in range(self.H):
                k, v = kc[ids, h * self.KV // self.H, off], vc[ids, h * self.KV // self.H, off]
                s = k @ q[b, h] * scale
                p = np.exp(s - s.max())
                size = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
                d = ((self.D + 4) + 10) * 2.0 ** -23 * size * 2 + 2.0 ** -22 + 2.0 ** -24
                A = (p / p.sum()) @ np.abs(v)
                tol = A * (2 * d + 2.0 ** -17 + 2 * (n + 320) * 2.0 ** -23)
                tol = tol + HALF_STEP[self.dtype] * (np.abs(want[b, h]) + tol) + 2.0 ** -25
                err = np.abs(got[b, h] - want[b, h])
                assert np.all(err <= tol), (b, h, float((err / tol).max()))


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 257]
SHAPES = [(1, 1, 64, 16), (8, 1, 256, 16), (6, 2, 96, 32), (4, 4, 128, 64), (16, 1, 192, 16), (10, 2, 64, 128),
          (17, 1, 128, 16), (40, 2, 64, 16), (3, 1, 96, 16), (2, 2, 192, 64)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,KV,D,page", SHAPES)
def test_lengths(H, KV, D, page, kind, dtype):
    b = Batch(EDGES, H, KV, D, page, dtype, kind, seed=H + D)
    b.check(b.run())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 700, 1001, 5000])
def test_one_sequence_split_and_joined(n, kind, dtype):
    import torch
    b = Batch([n], 8, 2, 128, 16, dtype, kind, seed=n)
    out = b.run()
    b.check(out)
    for limit in (n, 1, 0, 40, 4 * n, 1 << 20):   # how the work is split does not have to match the length
        b.check(b.run(max_len=limit))
    assert torch.equal(out, b.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("KV,D", [(2, 64), (16, 96), (1, 256), (8, 192)])
def test_one_workgroup_per_row(KV, D, kind):
    rng = np.random.default_rng(D)
    b = Batch([0, 1024, 1, 255, 1009] + list(rng.integers(0, 700, 11)), KV, KV, D, 32, "bf16", kind, seed=D)
    for max_len in (1024, 256, 1, 0):
        b.check(b.run(max_len=max_len))
    b.check(b.run(max_len=200, window=700, sinks=40), window=700, sinks=40)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (16, 4), (33, 1), (100, 40), (64, 64), (1000, 3),
                                          (31, 33)])
def test_window_and_sinks(window, sinks, kind):
    b = Batch(EDGES + [600, 1031], 4, 2, 64, 16, "fp16", kind, seed=window)
    b.check(b.run(window=window, sinks=sinks), window=window, sinks=sinks)
    b.check(b.run(window=window, sinks=sinks, max_len=1031), window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
def test_window_reads_no_hidden_page(kind):
    import torch
    b = Batch([500, 333, 64], 4, 1, 64, 16, "fp16", kind, seed=2)
    window, sinks = 70, 20
    want = b.run(window=window, sinks=sinks)
    for i, n in enumerate(b.lens):
        seen = set((od.visible(n, window, sinks) // 16).tolist())
        for p in range(b.table.shape[1]):
            if p not in seen:
                b.table[i, p] = -7 if p % 2 else 1 << 30
    assert torch.equal(b.run(window=window, sinks=sinks), want)
    # what is hidden inside visible pages may hold anything
    before = b.run(window=window, sinks=0)
    for i, n in enumerate(b.lens):
        first = n - window
        if first > 0 and first % 16:
            page = int(b.table[i, first // 16])
            b.cache[2][page, ..., :first % 16] = float("nan") if kind == "int8" else 255
            b.cache[3][page, ..., :first % 16] = float("nan") if kind == "int8" else 255
    assert torch.equal(b.run(window=window, sinks=0), before)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("entry", [-1, -(1 << 31), 1 << 20, (1 << 31) - 1])
def test_bad_page_poisons_its_sequence_only(entry, kind):
    import torch
    b = Batch([300, 300, 300, 40], 4, 2, 64, 16, "bf16", kind, seed=3)
    b.table[1, 7] = entry
    b.table[3, 2] = b.P
    for kw in ({}, dict(max_len=1)):
        out = b.run(**kw)
        assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3]).all())
        b.check(out, rows=[0, 2])


@pytest.mark.parametrize("kind", KINDS)
def test_length_beyond_the_table_and_negative(kind):
    import torch
    b = Batch([100, 100, 100, 100], 2, 1, 64, 16, "fp16", kind, seed=4)
    b.ld[1] = b.table.shape[1] * 16 + 1
    b.ld[2] = -5
    b.ld[3] = (1 << 31) - 1
    for kw in ({}, dict(window=10, sinks=2), dict(max_len=1 << 20)):
        out = b.run(**kw)
        assert bool(torch.isnan(out[1]).all()) and bool((out[2] == 0).all()) and bool(torch.isnan(out[3]).all())
    b.check(b.run(), rows=[0])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_peaked_and_flat_weights(kind, dtype):
    b = Batch([1500, 77], 4, 1, 128, 16, dtype, kind, seed=5, qscale=8.0)
    for scale in (1.0, 0.0, -0.3, 0.001):
        b.check(b.run(scale=scale), scale=scale)


@pytest.mark.parametrize("kind", KINDS)
def test_visible_nan_scale(kind):
    """A visible row that was stored as NaN makes its head's outputs NaN (a value's: in fp4 its 32 channels)."""
    import torch
    b = Batch([90, 90, 90], 4, 2, 64, 16, "fp16", kind, seed=7)
    nan = float("nan") if kind == "int8" else 255
    b.cache[2][int(b.table[0, 1]), 0, ..., 3] = nan            # a key of head 0
    if kind == "int8":
        b.cache[3][int(b.table[1, 2]), 1, 2] = nan             # a value of head 1
    else:
        b.cache[3][int(b.table[1, 2]), 1, 1, 2] = nan          # its channels 32 .. 63
    out = b.run()
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isfinite(out[1, :2]).all()) and bool(torch.isnan(out[1, 2:, 32:]).all())
    assert bool(torch.isnan(out[1, 2:, :32]).all()) == (kind == "int8")
    b.check(out, rows=[2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_strides_and_padding_untouched(offset, kind):
    """q a slice of a wider row, out a slice of a padded buffer, pages of codes and scales with gaps."""
    import torch
    H, KV, D, page = 6, 3, 64, 16
    b = Batch([100, 0, 40, 700], H, KV, D, page, "fp16", kind, seed=9)
    want = b.run()
    wide = torch.full((4, offset + H * D + 5), float("nan"), dtype=b.q.dtype, device="cuda")
    q = wide[:, offset:offset + H * D].unflatten(1, (H, D))
    q.copy_(b.q)
    cache = []
    for t in b.cache:
        big = torch.zeros((b.P, t[0].numel() + 64), dtype=t.dtype, device="cuda")
        big[:, :t[0].numel()] = t.flatten(1)
        cache.append(big[:, :t[0].numel()].view(t.shape))
    big = torch.full((5, offset + H * D + 3), 9.0, dtype=b.q.dtype, device="cuda")
    out = big[:4, offset:offset + H * D].unflatten(1, (H, D))
    bd.paged_attn_decode_quant(q, tuple(cache), b.table, b.ld, out=out)
    assert torch.equal(out, want)
    big[:4, offset:offset + H * D] = 9.0
    assert bool((big == 9.0).all())


@pytest.mark.parametrize("kind", KINDS)
def test_cache_past_32_bits(kind):
    import torch
    KV, D, page = 8, 128, 256
    b = Batch([500, 300], 16, KV, D, page, "bf16", kind, prefix=270, seed=10)
    row = D if kind == "int8" else D // 2
    P = (1 << 32) // (KV * row * page) + 3
    cache = bd.quant_pages(P, KV, page, D, kind)
    far = dict(zip(range(b.P), [P - 1, P - 2, P // 2 + 5, 1, P // 3, P - 7, 2, 9, P - 4, 4, 3]))
    assert len(far) == b.P
    for src, dst in far.items():
        for t, u in zip(b.cache, cache):
            u[dst] = t[src]
    move = lambda t: torch.tensor([[far.get(x, x) for x in r] for r in t.tolist()], dtype=torch.int32,  # noqa: E731
                                  device="cuda")
    table, pt = move(b.table), move(b.pt.view(1, -1)).view(-1)
    small = bd.paged_attn_decode_quant(b.q, b.cache, b.table, b.ld)
    assert torch.equal(bd.paged_attn_decode_quant(b.q, cache, table, b.ld), small)
    assert torch.equal(bd.paged_attn_shared(b.q, cache, pt, b.pl, table, b.ld), b.shared())


@pytest.mark.parametrize("kind", KINDS)
def test_graph_replays_with_growing_lengths(kind):
    import torch
    b = Batch([400, 900, 17], 8, 2, 128, 16, "bf16", kind, seed=11)
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


@pytest.mark.parametrize("kind", KINDS)
def test_side_stream_and_caller_workspace(kind):
    import torch
    b = Batch([20000], 4, 1, 64, 16, "fp16", kind, seed=12)
    want = b.run()
    need = bd.lib().w4a4_paged_attn_quant_workspace_bytes(1, 4, 1, 64, b.table.shape[1] * 16, 0, 0)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN bytes: nothing stale is read
    assert torch.equal(b.run(ws=ws), want)
    with pytest.raises(bd.W4A4Error, match="workspace"):
        b.run(ws=ws[:need - 256])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


# ---- behind a shared prefix ------------------------------------------------------------------------------------

PREFIXES = [0, 1, 15, 16, 17, 31, 32, 33, 64, 65, 127, 200, 513]


@pytest.mark.parametrize("kind", ["none", *KINDS])
@pytest.mark.parametrize("H,KV,D,page,B", [(1, 1, 64, 16, 1), (8, 1, 256, 16, 3), (6, 2, 96, 32, 7), (4, 4, 128, 64, 18),
                                           (16, 1, 192, 16, 2), (40, 2, 64, 16, 5), (8, 2, 128, 16, 40),
                                           (5, 1, 64, 32, 33)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_shared_prefix(H, KV, D, page, B, kind, dtype):
    lens = (EDGES * 3)[:B]
    for i, prefix in enumerate(PREFIXES):
        if (i + H + B) % 3 and prefix not in (0, 33):
            continue
        b = Batch(lens, H, KV, D, page, dtype, kind, prefix=prefix, seed=prefix + D)
        b.check(b.shared())


@pytest.mark.parametrize("kind", ["none", *KINDS])
def test_shared_hints_and_repeats(kind):
    import torch
    b = Batch([700, 0, 3, 64, 1000, 33], 8, 2, 128, 16, "fp16", kind, prefix=2500, seed=13)
    out = b.shared()
    b.check(out)
    for mp, ml in ((2500, 1000), (0, 0), (1, 1), (100000, 1 << 20), (64, 100000), (1 << 30, 0)):
        b.check(b.shared(max_prefix=mp, max_len=ml))
    assert torch.equal(out, b.shared())


@pytest.mark.parametrize("kind", ["none", *KINDS])
def test_shared_nothing_visible(kind):
    import torch
    b = Batch([0, 5, 0], 4, 2, 64, 16, "bf16", kind, prefix=0, seed=14)
    for n in (0, -3):
        b.pl.fill_(n)
        out = b.shared()
        b.check(out)
        assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
    out = bd.paged_attn_shared(b.q, b.cache, b.pt[:0], b.pl.zero_(), b.table, b.ld)     # no prefix table at all
    b.check(out)
    none = bd.paged_attn_shared(b.q[:0], b.cache, b.pt, b.pl, b.table[:0], b.ld[:0])
    assert none.shape == (0, 4, 64) and torch.cuda.is_available()


@pytest.mark.parametrize("kind", ["none", *KINDS])
def test_shared_bad_pages(kind):
    """A bad page of the prefix, or a prefix beyond its table, is everybody's; a bad page of one sequence its own."""
    import torch
    b = Batch([300, 0, 40, 20], 4, 2, 64, 16, "fp16", kind, prefix=200, seed=15)
    b.table[0, 3] = b.P
    b.ld[2] = b.table.shape[1] * 16 + 1
    out = b.shared()
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(out[2]).all())
    b.check(out, rows=[1, 3])
    for kw in ({}, dict(max_prefix=1), dict(max_prefix=100000)):
        b.pt[4] = -1
        assert bool(torch.isnan(b.shared(**kw)).all())
        b.pt[4] = 1 << 30
        assert bool(torch.isnan(b.shared(**kw)).all())
        b.pt[4] = 0
        for n in (b.pt.numel() * 16 + 1, (1 << 31) - 1):
            b.pl.fill_(n)
            assert bool(torch.isnan(b.shared(**kw)).all())
        b.pl.fill_(200)


@pytest.mark.parametrize("kind", ["none", *KINDS])
def test_shared_peaked_weights(kind):
    """The largest weight in the prefix for some sequences and in their own tokens for others, flat and reversed."""
    b = Batch([300, 77, 1], 4, 1, 128, 16, "bf16", kind, prefix=400, seed=16, qscale=8.0)
    for scale in (1.0, 0.0, -0.3):
        b.check(b.shared(scale=scale), scale=scale)


@pytest.mark.parametrize("kind", ["none", *KINDS])
def test_shared_graph_follows_the_lengths(kind):
    import torch
    b = Batch([400, 90, 0, 17], 8, 2, 64, 16, "fp16", kind, prefix=600, seed=17)
    full = list(b.lens)
    outs = [torch.empty_like(b.q) for _ in range(2)]
    b.shared()
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.shared(out=o)
        graphs.append(g)
    for cut, n in ((0, 600), (1, 599), (16, 31), (90, 0)):
        b.lens = [max(x - cut, 0) for x in full]
        b.prefix = n
        b.ld.copy_(torch.tensor(b.lens, dtype=torch.int32))
        b.pl.fill_(n)
        graphs[0].replay()
        graphs[1].replay()
        eager = b.shared()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager), cut
        b.check(eager)
        torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["none", *KINDS])
def test_shared_side_stream_workspace_and_strides(kind):
    import torch
    H, D = 4, 96
    b = Batch([20, 0, 700], H, 1, D, 16, "bf16", kind, prefix=1000, seed=18)
    want = b.shared()
    need = bd.lib().w4a4_paged_attn_shared_workspace_bytes(3, H, 1, D, b.pt.numel() * 16, b.table.shape[1] * 16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(b.shared(ws=ws), want)
    with pytest.raises(bd.W4A4Error, match="workspace"):
        b.shared(ws=ws[:need - 256])
    wide = torch.full((3, H * D + 7), float("nan"), dtype=b.q.dtype, device="cuda")
    q = wide[:, 3:3 + H * D].unflatten(1, (H, D))
    q.copy_(b.q)
    big = torch.full((4, H * D + 9), 9.0, dtype=b.q.dtype, device="cuda")
    out = big[:3, 1:1 + H * D].unflatten(1, (H, D))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bd.paged_attn_shared(q, b.cache, b.pt, b.pl, b.table, b.ld, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    big[:3, 1:1 + H * D] = 9.0
    assert bool((big == 9.0).all())
