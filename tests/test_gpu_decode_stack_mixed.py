"""Attention over the paged cache between linears that are quantized (W4A4, W8A8) or group-scaled: every linear
of the pass bit for bit or within its tolerance on its own recorded input, the attention's own steps against
the fp64 oracle."""
import numpy as np
import pytest

from oracle import decode as od
from w4a4_post_quantized_zigzag_amd import binding as bd
from w4a4_post_quantized_zigzag_amd.stack import LINEARS, Attention, DeviceStack, PagedCache

from parity_util import dev, host
from test_gpu_decode_stack import EPI, weights
from test_gpu_norm_rope import check as check_rope
from test_gpu_paged_attn import Batch
from test_gpu_w4g import check as check_linear

pytestmark = pytest.mark.gpu
GROUP, BLOCK, STEPS = 64, 128, 3
A = Attention(4, 2, 64, rot_dim=32, window=12, sinks=1)     # 256 attention channels beside 384 of the stack

MIXES = [dict(w4g=("qkv", "down"), w8=("o",)), dict(), dict(w8=LINEARS), dict(w4g=("o",), w8=("qkv", "down")),
         dict(w4g=("up",))]


def build(mix, layers=2, h=384, f=512, seed=1):
    W = weights(A, h, f, layers, seed=seed)
    return W, DeviceStack(W, BLOCK, STEPS, attention=A, group=GROUP, **mix)


def tables(ds, seed=2):
    """Scales of the right size, another per linear and step."""
    rng = np.random.default_rng(seed)
    return [{n: rng.uniform(0.3, 0.6, STEPS).astype(np.float32) for n in LINEARS} for _ in ds.layers]


def check_linears(ds, W, outs, step, mix):
    import torch
    epi = dict(none=bd.EPI_NONE, gelu=bd.EPI_GELU, residual=bd.EPI_RESIDUAL)
    for li, lw in enumerate(W):
        for n, (y, x, r) in zip(LINEARS, outs[4 * li:4 * li + 4]):
            if n in mix.get("w4g", ()):
                check_linear(y, x, *od.pack_w4g(lw[n], GROUP), GROUP, "fp16", EPI[n], r)
                continue
            lin = ds.layers[li][n]
            assert lin.bits == (8 if n in mix.get("w8", ()) else 4)
            x = x.contiguous()
            xq, xs = bd.rotate_quant_act(x, lin.perm, lin.rot, BLOCK, lin.table, STEPS, step, bits=lin.bits)
            want = bd.gemm(xq, xs, False, lin.wq, lin.w_scale, lin.K, epilogue=epi[EPI[n]], residual=r, bits=lin.bits)
            assert torch.equal(y, want), (li, n)


@pytest.mark.parametrize("mix", MIXES)
def test_every_call_of_the_pass(mix):
    layers, B, page = 2, 5, 16
    W, ds = build(mix)
    tl = tables(ds)
    ds.set_tables(tl)
    for li, layer in enumerate(ds.layers):
        for n in LINEARS:
            if n not in mix.get("w4g", ()):
                assert np.array_equal(host(layer[n].table), tl[li][n])
    cache = PagedCache(layers, A, B, pages=20, page_size=page, max_len=48)
    rng = np.random.default_rng(3)
    f64 = A.theta ** (-np.arange(0, A.rot_dim, 2) / A.rot_dim)
    for t in range(18):
        active = [t >= 3 * b for b in range(B)]
        cache.advance(active)
        outs, step = [], t % STEPS
        ds.run(dev(rng.standard_normal((B, 384)).astype(np.float16)), step, outputs=outs, cache=cache)
        if t not in (0, 7, 17):
            continue
        check_linears(ds, W, outs, step, mix)
        bufs, li = ds.bufs(B), layers - 1     # the last layer's attention buffers are still there
        q, k, v = outs[4 * li][0].view(B, -1, A.head_dim).split((A.heads, A.kv_heads, A.kv_heads), dim=1)
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


@pytest.mark.parametrize("mix", MIXES[:2])
def test_calibrating_pass_records_the_tables(mix):
    """run(calib=True) sets the step's entries of the quantized linears as the calibration of each linear's own
    input does, attention included; other steps stay."""
    import torch
    W, ds = build(mix)
    ds.set_tables(tables(ds))
    before = [{n: l[n].table.clone() for n in LINEARS if n not in mix.get("w4g", ())} for l in ds.layers]
    cache = PagedCache(2, A, 3, pages=6)
    cache.advance()
    outs = []
    X = dev(np.random.default_rng(5).standard_normal((3, 384)).astype(np.float16))
    ds.run(X, 1, calib=True, outputs=outs, cache=cache)
    for li, layer in enumerate(ds.layers):
        for n, (_, x, _) in zip(LINEARS, outs[4 * li:4 * li + 4]):
            if n in mix.get("w4g", ()):
                continue
            lin = layer[n]
            own = bd.calibrate_act_scale(x.contiguous(), lin.perm, lin.rot, BLOCK, bits=lin.bits)
            assert torch.equal(lin.table[1], own.view(())), (li, n)
            assert torch.equal(lin.table[[0, 2]], before[li][n][[0, 2]])


def test_graph_replayed_over_tokens():
    import torch
    mix = MIXES[0]
    W, ds = build(mix)
    ds.set_tables(tables(ds))
    rng = np.random.default_rng(6)
    caches = [PagedCache(2, A, 3, pages=9) for _ in range(2)]
    X = dev(rng.standard_normal((3, 384)).astype(np.float16))
    for c in caches:
        c.advance()
        ds.run(X, 2, cache=c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = ds.run(X, 2, cache=caches[0])
    for t in range(25):
        X.copy_(torch.from_numpy(rng.standard_normal((3, 384)).astype(np.float16)))
        for c in caches:
            c.advance([True, t % 2 == 0, t > 4])
        graph.replay()
        got = captured.clone()
        assert torch.equal(got, ds.run(X, 2, cache=caches[1])), t
        torch.cuda.synchronize()


def test_weights_and_norms_already_on_the_device():
    """Device tensors in place of numpy arrays, the norms in any float type and stride: the same stack."""
    import torch
    W = weights(A, 384, 512, 1, seed=8)
    for n in ("q_norm", "k_norm"):
        W[0][n] = W[0][n].astype(np.float16).astype(np.float32)
    there = {n: dev(w) for n, w in W[0].items()}
    there["q_norm"] = there["q_norm"].half()
    there["k_norm"] = torch.stack((there["k_norm"], there["k_norm"]), 1)[:, 0]
    X = dev(np.random.default_rng(9).standard_normal((2, 384)).astype(np.float16))
    outs = []
    for w in (W, [there]):
        ds = DeviceStack(w, BLOCK, 1, w4g=LINEARS, group=GROUP, attention=A)
        cache = PagedCache(1, A, 2, pages=2)
        cache.advance()
        outs.append(ds.run(X, 0, cache=cache).clone())
    assert torch.equal(*outs)
