"""The single-token calls beside each other: on two streams at once, in two graphs, on shared pages and
slots. Every result is compared bit for bit with the same call made alone, which the parity tests of
each call check against the oracle."""
import numpy as np
import pytest

from w4a4_post_quantized_zigzag_amd import binding as bd

from parity_util import dev, host
from test_gpu_norm_rope import f64, freqs, make
from test_gpu_paged_attn import Batch

pytestmark = pytest.mark.gpu


class Job:
    """A linear, a norm + rotation with append and an attention of one batch, on memory of their own."""

    def __init__(self, lens, H, KV, D, dtype, seed):
        import torch
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.b = Batch(lens, H, KV, D, 16, dtype, seed=seed)
        self.rows = make(B, H, KV, D, dtype, seed=seed)
        self.freq = dev(freqs(D))
        self.kc = torch.zeros((B, KV, 16, D), dtype=self.b.q.dtype, device="cuda")
        self.vc = torch.zeros_like(self.kc)
        self.slots = dev((np.arange(B) * 16 + rng.integers(0, 16, B)).astype(np.int64))
        K, N = H * D, 1000
        self.x = dev(rng.standard_normal((B, K)).astype(np.float32)).to(self.b.q.dtype)
        self.wt, self.ws = bd.pack_weights_w4g(dev(rng.standard_normal((N, K)).astype(np.float32)), 64)

    def run(self):
        q, k, v, wq, wk, pos = self.rows
        qo = bd.qk_norm_rope_append(q, k, v, wq, wk, self.freq, pos, self.kc, self.vc, self.slots)
        return [bd.gemv_w4g(self.x, self.wt, self.ws), qo, self.b.run(), self.b.run(window=100, sinks=3)]

    def state(self, outs):
        return [host(t.float()) for t in (*outs, self.kc, self.vc)]


def jobs():
    return [Job([3000, 0, 17, 5001, 640], 8, 2, 128, "bf16", 1), Job([900, 33, 1], 6, 1, 96, "fp16", 2)]


def same(a, b):
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)


def test_two_streams_at_once():
    import torch
    js = jobs()
    alone = [j.state(j.run()) for j in js]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in js]
    outs = []
    for _ in range(10):
        for j, s in zip(js, streams):
            with torch.cuda.stream(s):
                outs.append((j, j.run()))
    torch.cuda.synchronize()
    for j, o in outs:
        same(j.state(o), alone[js.index(j)])


def test_two_graphs_replayed_in_turn_and_at_once():
    import torch
    js = jobs()
    alone = [j.state(j.run()) for j in js]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for j in js:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(j.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in js]
    for turn in range(4):
        for j, o in zip(js, outs):
            for t in (*o, j.kc, j.vc):
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s if turn % 2 else torch.cuda.current_stream()):
                g.replay()
        torch.cuda.synchronize()
        for j, o, a in zip(js, outs, alone):
            same(j.state(o), a)
            same(j.state(j.run()), a)  # eager work between the replays
            torch.cuda.synchronize()


def test_two_rows_with_one_slot():
    import torch
    q, k, v, wq, wk, pos = make(6, 2, 2, 64, "fp16", seed=3)
    kc = torch.zeros((2, 2, 16, 64), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = dev(np.array([5, 20, 5, 20, 5, 31], np.int64))
    ko = torch.empty((6, 2, 64), dtype=torch.float16, device="cuda")
    bd.qk_norm_rope_append(q, k, v, wq, wk, dev(freqs(64)), pos, kc, vc, slots, k_out=ko)
    for s in (5, 20, 31):
        rows = [m for m in range(6) if int(slots[m]) == s]
        for cache, src in ((kc, ko), (vc, v)):
            got = f64(cache[s // 16, :, s % 16])
            assert np.all(np.any([got == f64(src[m]) for m in rows], axis=0))
    used = np.zeros((2, 16), bool)
    used[0, 5] = used[1, 4] = used[1, 15] = True
    for cache in (kc, vc):
        assert not np.any(f64(cache).transpose(0, 2, 1, 3)[~used])


def test_sequences_that_share_pages():
    import torch
    b = Batch([1500, 1500, 700], 8, 2, 64, 32, "bf16", seed=4)
    b.table[1] = b.table[0]
    b.table[2, :22] = b.table[0, :22]
    b.q[1] = b.q[0]
    out = b.run()
    assert torch.equal(out[0], out[1])
    b.check(out)
