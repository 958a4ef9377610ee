"""The single-token path of the stack: group-scaled linears, norm + rotation + append and attention over
the paged cache run together, token by token.

Teacher-forced: every call of the pass is checked against the fp64 oracle on the device's own inputs to it,
with the tolerances of the per-operator tests. Free-running: the whole chain against the oracle's own chain,
with the stack's end-to-end tolerances. Also captured into one HIP graph and replayed token after token."""
import numpy as np
import pytest

from oracle import decode as od
from w4a4_post_quantized_zigzag_amd import binding as bd
from w4a4_post_quantized_zigzag_amd import inputs
from w4a4_post_quantized_zigzag_amd.stack import LINEARS, Attention, DeviceStack, PagedCache

from parity_util import check_y_tolerance, dev, host
from test_gpu_norm_rope import check as check_rope
from test_gpu_paged_attn import Batch
from test_gpu_w4g import check as check_linear

pytestmark = pytest.mark.gpu
GROUP = 64
EPI = dict(qkv="none", o="residual", up="gelu", down="residual")


def weights(A, h, f, layers, seed):
    rng = np.random.default_rng(seed)
    n = (A.heads + 2 * A.kv_heads) * A.head_dim
    shapes = dict(qkv=(n, h), o=(h, A.heads * A.head_dim), up=(f, h), down=(h, f))
    out = []
    for _ in range(layers):
        lw = {k: rng.normal(0, 0.05, s).astype(np.float16) for k, s in shapes.items()}
        lw["q_norm"] = (1 + 0.2 * rng.standard_normal(A.head_dim)).astype(np.float32)
        lw["k_norm"] = (1 + 0.2 * rng.standard_normal(A.head_dim)).astype(np.float32)
        out.append(lw)
    return out


SPECS = [Attention(4, 2, 64), Attention(6, 1, 64, rot_dim=32, interleaved=True, window=9, sinks=2),
         Attention(2, 2, 128, rot_dim=0)]


@pytest.mark.parametrize("A", SPECS)
def test_every_call_of_the_pass(A):
    h, f, layers, B, page = 256, 512, 2, 5, 16
    W = weights(A, h, f, layers, seed=A.heads)
    packed = [{n: od.pack_w4g(lw[n], GROUP) for n in LINEARS} for lw in W]
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A)
    cache = PagedCache(layers, A, B, pages=20, page_size=page, max_len=48)
    rng = np.random.default_rng(1)
    rot = A.head_dim if A.rot_dim is None else A.rot_dim
    f64 = A.theta ** (-np.arange(0, rot, 2) / rot) if rot else None
    for t in range(20):
        active = [t >= 3 * b for b in range(B)]      # sequences start at different times
        cache.advance(active)
        outs = []
        ds.run(dev(rng.standard_normal((B, h)).astype(np.float16)), 0, outputs=outs, cache=cache)
        if t not in (0, 8, 19):
            continue
        bufs = ds.bufs(B)
        for li in range(layers):
            for n, (y, x, r) in zip(LINEARS, outs[4 * li:4 * li + 4]):
                codes, s = packed[li][n]
                check_linear(y, x, codes, s, GROUP, "fp16", EPI[n], r)
        # the last layer's attention buffers are still there
        li = layers - 1
        qkv = outs[4 * li][0].view(B, -1, A.head_dim)
        q, k, v = qkv.split((A.heads, A.kv_heads, A.kv_heads), dim=1)
        check_rope(bufs.q, q, ds.norms[li][0], A.eps, f64, cache.positions, A.interleaved, "fp16")
        slots = host(cache.slots)
        for b in range(B):
            if active[b]:
                p, o = slots[b] // page, slots[b] % page
                check_rope(cache.k[li][p:p + 1, :, o], k[b:b + 1], ds.norms[li][1], A.eps, f64,
                           cache.positions[b:b + 1], A.interleaved, "fp16")
                assert np.array_equal(host(cache.v[li][p, :, o]), host(v[b]))
        att = Batch.__new__(Batch)
        att.lens, att.H, att.KV, att.D, att.page, att.dtype = (host(cache.lens).tolist(), A.heads, A.kv_heads,
                                                               A.head_dim, page, "fp16")
        att.q, att.kc, att.vc, att.table = bufs.q, cache.k[li], cache.v[li], cache.table
        att.check(bufs.att, window=A.window, sinks=A.sinks)


def oracle_token(W, packed, A, X, kv, positions, active, freqs):
    """One pass of the chain in fp64 with fp16 roundings where the device stores fp16."""
    r16 = lambda a: a.astype(np.float16).astype(np.float64)  # noqa: E731
    cur = X.astype(np.float64)
    B = X.shape[0]
    for li, lw in enumerate(W):
        lin = lambda n, x, res=None: r16(od.linear_w4g(x, *packed[li][n], EPI[n], res)[0])  # noqa: E731
        qkv = lin("qkv", cur).reshape(B, -1, A.head_dim)
        q = r16(od.norm_rope(qkv[:, :A.heads], lw["q_norm"], A.eps, freqs, positions, A.interleaved))
        k = r16(od.norm_rope(qkv[:, A.heads:A.heads + A.kv_heads], lw["k_norm"], A.eps, freqs, positions,
                             A.interleaved))
        att = np.zeros((B, A.heads, A.head_dim))
        for b in range(B):
            if active[b]:
                kv[li][b].append((k[b], qkv[b, A.heads + A.kv_heads:]))
            past = kv[li][b]
            j = od.visible(len(past), A.window, A.sinks)
            for hd in range(A.heads if j.size else 0):
                kh = hd * A.kv_heads // A.heads
                s = np.array([past[i][0][kh] @ q[b, hd] for i in j]) * A.head_dim ** -0.5
                p = np.exp(s - s.max())
                att[b, hd] = (p / p.sum()) @ np.array([past[i][1][kh] for i in j])
        h2 = lin("o", r16(att).reshape(B, -1), cur)
        cur = lin("down", lin("up", h2), h2)
    return cur


def test_free_running_chain():
    A = SPECS[1]
    h, f, layers, B = 256, 512, 2, 3
    W = weights(A, h, f, layers, seed=4)
    packed = [{n: od.pack_w4g(lw[n], GROUP) for n in LINEARS} for lw in W]
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A)
    cache = PagedCache(layers, A, B, pages=8, page_size=16)
    kv = [[[] for _ in range(B)] for _ in range(layers)]
    rng = np.random.default_rng(2)
    rot = A.rot_dim
    freqs = A.theta ** (-np.arange(0, rot, 2) / rot)
    for t in range(18):
        active = [True, t % 2 == 0, t >= 5]
        cache.advance(active)
        X = rng.standard_normal((B, h)).astype(np.float16)
        got = host(ds.run(dev(X), 0, cache=cache))
        want = oracle_token(W, packed, A, X, kv, host(cache.positions), active, freqs)
        check_y_tolerance(got, want)
    cache.release(0)
    assert len(cache._free) == 8 - 2                   # sequences 1 and 2 hold a page each


def test_graph_replayed_over_tokens():
    import torch
    A = SPECS[0]
    h, f, layers, B = 256, 512, 2, 4
    W = weights(A, h, f, layers, seed=5)
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A)
    rng = np.random.default_rng(3)
    X = torch.empty((B, h), dtype=torch.float16, device="cuda")
    caches = [PagedCache(layers, A, B, pages=16, page_size=16, max_len=64) for _ in range(2)]
    first = rng.standard_normal((B, h)).astype(np.float16)
    X.copy_(torch.from_numpy(first))
    for c in caches:
        c.advance()
        ds.run(X, 0, cache=c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ds.run(X, 0, cache=caches[0])
    for t in range(35):
        X.copy_(torch.from_numpy(rng.standard_normal((B, h)).astype(np.float16)))
        for c in caches:
            c.advance()
        graph.replay()
        got = captured.clone()
        assert torch.equal(got, ds.run(X, 0, cache=caches[1])), t
        torch.cuda.synchronize()
    for a, b in zip(caches[0].k + caches[0].v, caches[1].k + caches[1].v):
        assert torch.equal(a, b)


def test_group_linears_beside_quantized_ones():
    """Only some linears group-scaled, no attention: the others give what their own W4A4 / W8A8 calls
    give on the same inputs, bit for bit."""
    import torch
    Ls, h, f, M, T = 2, 256, 1024, 40, 2
    W = inputs.stack_weights(layers=Ls, hidden=h, ffn=f)
    Ac = inputs.stack_activations(M=M, hidden=h, steps=T, calib=2)
    ds = DeviceStack(W, 128, T, w8=("o",), w4g=("qkv", "down"), group=128)
    ds.calibrate(Ac["X_calib"])
    outs = []
    ds.run(dev(Ac["X_steps"][1]), 1, outputs=outs)
    for li in range(Ls):
        for n, (y, x, r) in zip(LINEARS, outs[4 * li:4 * li + 4]):
            if n in ("qkv", "down"):
                codes, s = od.pack_w4g(W[li][n].astype(np.float32), 128)
                check_linear(y, x, codes, s, 128, "fp16", EPI[n], r)
            else:
                lin, epi = ds.layers[li][n], {"up": bd.EPI_GELU, "o": bd.EPI_RESIDUAL}[n]
                xq, xs = bd.rotate_quant_act(x, lin.perm, lin.rot, 128, lin.table, T, 1, bits=lin.bits)
                want = bd.gemm(xq, xs, False, lin.wq, lin.w_scale, lin.K, epilogue=epi, residual=r,
                               bits=lin.bits)
                assert torch.equal(y, want), (li, n)


def test_refusals():
    A = SPECS[0]
    W = weights(A, 256, 512, 1, seed=6)
    with pytest.raises(ValueError, match="qkv rows"):
        DeviceStack(W, 128, 1, w4g=LINEARS, attention=Attention(4, 1, 64))
    with pytest.raises(ValueError, match="different linears"):
        DeviceStack(W, 128, 1, w8=("o",), w4g=("o",))
    ds = DeviceStack(W, 128, 1, w4g=LINEARS, group=GROUP, attention=A)
    X = dev(np.zeros((2, 256), np.float16))
    with pytest.raises(ValueError, match="cache"):
        ds.run(X, 0)
    cache = PagedCache(1, A, 3, pages=2, page_size=16)
    with pytest.raises(ValueError, match="rows"):
        ds.run(X, 0, cache=cache)
    with pytest.raises(ValueError, match="set_tables"):
        ds.calibrate([])
    with pytest.raises(RuntimeError, match="no free pages"):
        cache.advance()
    small = PagedCache(1, A, 1, pages=2, page_size=16, max_len=1)
    small.advance()
    with pytest.raises(RuntimeError, match="max_len"):
        small.advance()
