"""The stack's serving path run together: a cache in 16, 8 or 4 bits, a prefix that all sequences share, and low-rank
adapters that differ from row to row, token by token.

Teacher-forced: every call of a pass is checked against the fp64 oracle on the device's own inputs to it, with the
tolerances of the per-operator tests (a quantized cache's new rows bit for bit against its two halves). Free-running: the
whole chain over a 16-bit cache against the oracle's own chain, with the stack's end-to-end tolerances. Captured into one
HIP graph and replayed while lengths and ids change, against the same calls made one by one, bit for bit."""
import numpy as np
import pytest

from oracle import decode as od
from oracle import served as osv
from w4a4_post_quantized_zigzag_amd import binding as bd
from w4a4_post_quantized_zigzag_amd.stack import LINEARS, Attention, DeviceStack, PagedCache

from parity_util import check_y_tolerance, dev, host
from test_gpu_adapter import Case
from test_gpu_decode_stack import EPI, GROUP, weights
from test_gpu_kv_attn import Batch
from test_gpu_w4g import check as check_linear

pytestmark = pytest.mark.gpu
KINDS = ["fp16", "int8", "fp4"]


def make_adapters(W, n, seed, names=LINEARS, R=16):
    rng = np.random.default_rng(seed)
    out = []
    for lw in W:
        layer = {}
        for name in names:
            N, K = lw[name].shape
            layer[name] = ((rng.standard_normal((n, R, K)) * K ** -0.5).astype(np.float16),
                           (0.3 * rng.standard_normal((n, N, R))).astype(np.float16),
                           (0.5 + rng.random(n)).astype(np.float32))
        out.append(layer)
    return out


def values(cache, li):
    """The fp64 values (keys, values) of layer li's whole cache [pages, kv, page, D]."""
    c = cache.kv[li]
    if cache.kind == "fp16":
        return [host(t).astype(np.float64) for t in c]
    if cache.kind == "int8":
        return [osv.values_int8(host(c[i]), host(c[2 + i])) for i in (0, 1)]
    out = []
    for i in (0, 1):
        packed = host(c[i])
        codes = np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)
        out.append(osv.values_fp4(codes, host(c[2 + i]).transpose(0, 1, 3, 2)))
    return out


def check_attention(cache, li, A, q, out):
    att = Batch.__new__(Batch)
    att.lens, att.H, att.KV, att.D, att.page, att.dtype = (host(cache.lens).tolist(), A.heads, A.kv_heads, A.head_dim,
                                                           cache.page_size, "fp16")
    att.q, att.values, att.table, att.pt, att.prefix = (q, values(cache, li), cache.table, cache.prefix_table,
                                                        int(cache.prefix_len[0]))
    att.check(out, window=A.window, sinks=A.sinks)


SPECS = [(Attention(4, 2, 64), 0, 0), (Attention(6, 1, 64, rot_dim=32, interleaved=True, window=9, sinks=2), 0, 0),
         (Attention(4, 2, 64), 21, 40), (Attention(10, 2, 128, rot_dim=0), 33, 33)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("A,prefix,most", SPECS)
def test_every_call_of_the_pass(A, prefix, most, kind):
    import torch
    h, f, layers, B, page, n = 256, 512, 2, 5, 16, 3
    W = weights(A, h, f, layers, seed=A.heads)
    ad = make_adapters(W, n, seed=1, names=("qkv", "down", "up") if A.window else LINEARS)
    packed = [{name: od.pack_w4g(lw[name], GROUP) for name in LINEARS} for lw in W]
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A, adapters=ad)
    cache = PagedCache(layers, A, B, pages=20, page_size=page, max_len=48, kv=kind, max_prefix=most)
    rng = np.random.default_rng(1)
    ids = dev(np.array([0, 2, -1, 1, 0], np.int32))
    for t in range(prefix + 12):
        active = [t - prefix >= 2 * b for b in range(B)]   # sequences start at different times
        if t < prefix:
            cache.advance_prefix(row=t % B)
        else:
            cache.advance(active)
        outs = []
        X = dev(rng.standard_normal((B, h)).astype(np.float16))
        ds.run(X, 0, outputs=outs, cache=cache, adapters=ids)
        if t not in (0, prefix, prefix + 11):
            continue
        bufs = ds.bufs(B)
        for li in range(layers):
            for name, (y, x, r) in zip(LINEARS, outs[4 * li:4 * li + 4]):
                if name not in ad[li]:
                    check_linear(y, x, *packed[li][name], GROUP, "fp16", EPI[name], r)
                    continue
                lin, c = ds.layers[li][name], Case.__new__(Case)
                c.dtype, c.X, c.res, c.ids = "fp16", x, r if r is not None else y, ids
                c.A, c.B, c.scale = ds.adapters[li][name]
                c.Y = bd.gemv_w4g(x, lin.wt, lin.w_scale)
                check_linear(c.Y, x, *packed[li][name], GROUP, "fp16")
                c.check(y, EPI[name])
        # the last layer's attention buffers are still there
        li = layers - 1
        qkv = outs[4 * li][0].view(B, -1, A.head_dim)
        q, k, v = qkv.split((A.heads, A.kv_heads, A.kv_heads), dim=1)
        qo, ko = bd.qk_norm_rope(q, k, *ds.norms[li], ds.inv_freq, cache.positions, eps=A.eps,
                                 interleaved=A.interleaved)
        assert torch.equal(bufs.q, qo)
        seen = cache.slots >= 0
        assert int(seen.sum()) == (1 if t < prefix else sum(active))
        other = PagedCache(1, A, B, pages=20, page_size=page, kv=kind)
        other.write(0, ko, v, cache.slots)
        for got, want in zip(cache.read(li, cache.slots), other.read(0, cache.slots)):
            assert torch.equal(got, want)
        check_attention(cache, li, A, bufs.q, bufs.att)


def oracle_token(W, packed, ad, ids, A, X, kv, positions, owner, freqs):
    """One pass of the chain in fp64 with fp16 roundings where the device stores fp16. kv: per layer, per row, the tokens
    it sees. owner[b]: the lists that row b's new token joins."""
    r16 = lambda a: a.astype(np.float16).astype(np.float64)  # noqa: E731
    cur, B = X.astype(np.float64), X.shape[0]
    for li, lw in enumerate(W):
        def lin(name, x, res=None):
            y = r16(od.linear_w4g(x, *packed[li][name], "none", None)[0])
            return r16(osv.adapter_add(y, x, *ad[li][name][:2], ids, ad[li][name][2], EPI[name], res)[0])
        qkv = lin("qkv", cur).reshape(B, -1, A.head_dim)
        q = r16(od.norm_rope(qkv[:, :A.heads], lw["q_norm"], A.eps, freqs, positions, A.interleaved))
        k = r16(od.norm_rope(qkv[:, A.heads:A.heads + A.kv_heads], lw["k_norm"], A.eps, freqs, positions, A.interleaved))
        att = np.zeros((B, A.heads, A.head_dim))
        for b in range(B):
            for row in owner[b]:
                kv[li][row].append((k[b], qkv[b, A.heads + A.kv_heads:]))
        for b in range(B):
            past = kv[li][b]
            for hd in range(A.heads if past else 0):
                kh = hd * A.kv_heads // A.heads
                s = np.array([p[0][kh] @ q[b, hd] for p in past]) * A.head_dim ** -0.5
                p = np.exp(s - s.max())
                att[b, hd] = (p / p.sum()) @ np.array([p[1][kh] for p in past])
        h2 = lin("o", r16(att).reshape(B, -1), cur)
        cur = lin("down", lin("up", h2), h2)
    return cur


def test_free_running_chain():
    A = Attention(4, 2, 64)
    h, f, layers, B, n, prefix = 256, 512, 2, 3, 2, 19
    W = weights(A, h, f, layers, seed=4)
    ad = make_adapters(W, n, seed=5)
    packed = [{name: od.pack_w4g(lw[name], GROUP) for name in LINEARS} for lw in W]
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A, adapters=ad)
    cache = PagedCache(layers, A, B, pages=8, page_size=16, max_len=32, max_prefix=32)
    kv = [[[] for _ in range(B)] for _ in range(layers)]
    rng = np.random.default_rng(2)
    ids = [1, -1, 0]
    freqs = A.theta ** (-np.arange(0, A.head_dim, 2) / A.head_dim)
    for t in range(prefix + 9):
        if t < prefix:
            cache.advance_prefix(1)
            owner, of = [[], list(range(B)), []], [1]           # the row that is a token of every sequence
        else:
            active = [True, t % 2 == 0, t >= prefix + 4]
            cache.advance(active)
            owner, of = [[b] if active[b] else [] for b in range(B)], range(B)
        X = rng.standard_normal((B, h)).astype(np.float16)
        got = host(ds.run(dev(X), 0, cache=cache, adapters=dev(np.array(ids, np.int32))))
        want = oracle_token(W, packed, ad, ids, A, X, kv, host(cache.positions), owner, freqs)
        check_y_tolerance(got[list(of)], want[list(of)])
    cache.release(0)
    assert len(cache._free) == 8 - 2 - 2                       # the prefix's two pages, one of each other sequence
    with pytest.raises(RuntimeError, match="go on"):
        cache.release_prefix()
    cache.release(1), cache.release(2)
    cache.release_prefix()
    assert len(cache._free) == 8 and int(cache.prefix_len[0]) == 0


@pytest.mark.parametrize("kind,prefix", [("int8", 0), ("fp4", 0), ("fp16", 17), ("int8", 17), ("fp4", 40)])
def test_graph_replayed_over_tokens(kind, prefix):
    import torch
    A = Attention(4, 2, 64)
    h, f, layers, B = 256, 512, 2, 4
    W = weights(A, h, f, layers, seed=5)
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A, adapters=make_adapters(W, 5, seed=6))
    rng = np.random.default_rng(3)
    X = torch.zeros((B, h), dtype=torch.float16, device="cuda")
    ids = torch.zeros(B, dtype=torch.int32, device="cuda")
    caches = [PagedCache(layers, A, B, pages=20, page_size=16, max_len=64, kv=kind, max_prefix=prefix) for _ in range(2)]
    ds.run(X, 0, cache=caches[0], adapters=ids)                # nothing to append yet: slots are -1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ds.run(X, 0, cache=caches[0], adapters=ids)
    for t in range(prefix + 24):
        X.copy_(torch.from_numpy(rng.standard_normal((B, h)).astype(np.float16)))
        ids.copy_(torch.from_numpy(rng.integers(-1, 6, B).astype(np.int32)))
        for c in caches:
            c.advance_prefix() if t < prefix else c.advance()
        graph.replay()
        got = captured.clone()
        assert torch.equal(got, ds.run(X, 0, cache=caches[1], adapters=ids)), t
        torch.cuda.synchronize()
    for a, b in zip(caches[0].kv, caches[1].kv):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("kind", KINDS)
def test_rows_brought_from_elsewhere(kind):
    """extend + write against tokens that run() appended one by one: the same cache, and read() gives it back."""
    import torch
    A = Attention(4, 2, 128)
    h, B, prefix, own = 256, 2, 23, 18
    W = weights(A, h, 512, 1, seed=8)
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A)
    make = lambda: PagedCache(1, A, B, pages=12, page_size=16, max_len=48, kv=kind, max_prefix=32)  # noqa: E731
    a, b = make(), make()
    rng = np.random.default_rng(9)
    X = [dev(rng.standard_normal((B, h)).astype(np.float16)) for _ in range(prefix + own + 1)]
    lin = ds.layers[0]["qkv"]

    def rows(row, ts):
        qkv = bd.gemv_w4g(torch.stack([X[t][row] for t in ts]), lin.wt, lin.w_scale).view(len(ts), -1, A.head_dim)
        q, k, v = qkv.split((A.heads, A.kv_heads, A.kv_heads), dim=1)
        at = torch.tensor(list(ts), dtype=torch.int64, device="cuda")
        return bd.qk_norm_rope(q, k, *ds.norms[0], ds.inv_freq, at)[1], v.contiguous()

    for t in range(prefix + own):
        a.advance_prefix() if t < prefix else a.advance()
        ds.run(X[t], 0, cache=a)
    b.write(0, *rows(0, range(prefix)), b.extend(None, prefix))
    for row in range(B):
        b.write(0, *rows(row, range(prefix, prefix + 5)), b.extend(row, 5))
        b.write(0, *rows(row, range(prefix + 5, prefix + own)), b.extend(row, own - 5))
    for row in (None, 0, 1):
        for got, want in zip(b.read(0, b.slots_of(row)), a.read(0, a.slots_of(row))):
            assert got.shape[0] == prefix + (0 if row is None else own)
            assert torch.equal(got, want) and got.any()
    for c in (a, b):
        c.advance()
    assert torch.equal(a.positions, b.positions) and torch.equal(a.lens, b.lens)
    assert int(a.positions[0]) == prefix + own
    assert torch.equal(ds.run(X[-1], 0, cache=a), ds.run(X[-1], 0, cache=b))
    gone = torch.tensor([-1, int(b.slots_of(0)[3])], device="cuda")
    k, v = b.read(0, gone)
    assert not k[0].any() and not v[0].any() and k[1].any()
    assert b.extend(0, 0).shape == (0,)


def test_adapters_beside_quantized_linears():
    """W4A4 and W8A8 linears, no attention: each is its own call without an epilogue, then the adapters."""
    import torch
    from w4a4_post_quantized_zigzag_amd import inputs
    Ls, h, f, M, T = 2, 256, 1024, 40, 2
    W = inputs.stack_weights(layers=Ls, hidden=h, ffn=f)
    Ac = inputs.stack_activations(M=M, hidden=h, steps=T, calib=2)
    ad = make_adapters(W, 3, seed=7, names=("qkv", "o", "down"), R=8)
    ds = DeviceStack(W, 128, T, w8=("o",), adapters=ad)
    plain = DeviceStack(W, 128, T, w8=("o",), w4g=(), adapters=[{}] * Ls)
    ds.calibrate(Ac["X_calib"])
    plain.calibrate(Ac["X_calib"])
    X = dev(Ac["X_steps"][1])
    ids = dev(np.arange(M, dtype=np.int32) % 4 - 1)
    assert torch.equal(ds.run(X, 1), plain.run(X, 1))                # without ids: the linears as they are
    assert torch.equal(ds.run(X, 1, adapters=torch.full_like(ids, 3)).isfinite(), X.isfinite())
    outs = []
    ds.run(X, 1, outputs=outs, adapters=ids)
    for li in range(Ls):
        for name, (y, x, r) in zip(LINEARS, outs[4 * li:4 * li + 4]):
            lin, epi = ds.layers[li][name], {"none": bd.EPI_NONE, "gelu": bd.EPI_GELU, "residual": bd.EPI_RESIDUAL}[EPI[name]]
            xq, xs = bd.rotate_quant_act(x, lin.perm, lin.rot, 128, lin.table, T, 1, bits=lin.bits)
            has = name in ad[li]
            base = bd.gemm(xq, xs, False, lin.wq, lin.w_scale, lin.K, epilogue=bd.EPI_NONE if has else epi,
                           residual=None if has else r, bits=lin.bits)
            want = bd.adapter_add(base, x, *ds.adapters[li][name][:2], ids, ds.adapters[li][name][2], epilogue=epi,
                                  residual=r) if has else base
            assert torch.equal(y, want), (li, name)


def test_refusals():
    import torch
    A = Attention(4, 2, 64)
    W = weights(A, 256, 512, 2, seed=6)
    ad = make_adapters(W, 3, seed=7)
    build = lambda a: DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A, adapters=a)  # noqa: E731
    with pytest.raises(ValueError, match="layers"):
        build(ad[:1])
    with pytest.raises(ValueError, match="linears are"):
        build([{"qvk": ad[0]["qkv"]}, {}])
    with pytest.raises(ValueError, match="must be A"):
        build([{"o": ad[0]["down"]}, {}])
    with pytest.raises(ValueError, match="must be A"):
        build([{"o": (ad[0]["o"][0][:, :12], ad[0]["o"][1][:, :, :12])}, {}])
    with pytest.raises(ValueError, match="a scale"):
        build([{"o": (*ad[0]["o"][:2], np.ones(2, np.float32))}, {}])
    with pytest.raises(ValueError, match="same for all"):
        build([{"o": ad[0]["o"]}, {"o": tuple(t[:2] for t in ad[1]["o"])}])
    with pytest.raises(ValueError, match="kv must be"):
        PagedCache(1, A, 1, pages=2, kv="int4")
    with pytest.raises(ValueError, match="without a window"):
        PagedCache(1, Attention(4, 2, 64, window=8), 1, pages=2, max_prefix=16)
    with pytest.raises(ValueError, match="multiple of 32"):
        PagedCache(1, Attention(4, 2, 80), 1, pages=2, kv="fp4")
    X = torch.zeros((2, 256), dtype=torch.float16, device="cuda")
    cache = PagedCache(2, A, 2, pages=4, max_len=32, max_prefix=20)
    bare = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A)
    with pytest.raises(ValueError, match="has none"):
        bare.run(X, 0, cache=cache, adapters=torch.zeros(2, dtype=torch.int32, device="cuda"))
    ds = build(ad)
    for ids in (torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
                torch.zeros(2, dtype=torch.int32)):
        with pytest.raises((ValueError, TypeError)):
            ds.run(X, 0, cache=cache, adapters=ids)
    windowed = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=Attention(4, 2, 64, window=8))
    with pytest.raises(ValueError, match="without a window"):
        windowed.run(X, 0, cache=cache)
    with pytest.raises(RuntimeError, match="max_prefix"):
        cache.extend(None, 21)
    assert len(cache._free) == 4                               # a refusal takes no page
    with pytest.raises(IndexError):
        cache.extend(2, 1)
    with pytest.raises(IndexError):
        cache.advance_prefix(2)
    assert cache._prefix == 0
    with pytest.raises(ValueError, match="tokens"):
        cache.extend(0, -1)
    cache = PagedCache(2, A, 2, pages=4, max_len=32, max_prefix=20)
    cache.extend(None, 20)
    cache.extend(0, 16)
    with pytest.raises(RuntimeError, match="complete"):
        cache.advance_prefix()
    with pytest.raises(RuntimeError, match="max_len"):
        cache.extend(0, 17)
    with pytest.raises(RuntimeError, match="no free pages"):
        cache.advance([True, True])
    assert cache._len == [16, 0] and len(cache._free) == 1
    none = PagedCache(2, A, 2, pages=4)
    with pytest.raises(RuntimeError, match="max_prefix 0"):
        none.advance_prefix()
