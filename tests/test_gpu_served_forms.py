"""Every form of the serving kernels at the sizes where one gives way to another: how many rows a prefix's waves share, more
tiles than one look at the page table covers, shared memory past 64 KB, and the adapters' walks and parts. Oracle and
tolerances as in test_gpu_kv_attn.py and test_gpu_adapter.py."""
import numpy as np
import pytest

from parity_util import dev
from test_gpu_adapter import Case
from test_gpu_kv_attn import Batch
from test_gpu_norm_rope import tdt

pytestmark = pytest.mark.gpu
ALL = ["none", "int8", "fp4"]


# rows a key head: 2, 3 and 4 tiles of 16 (two, two and four waves on rows), 5 and 9 (two tiles a wave)
@pytest.mark.parametrize("B,group", [(9, 2), (33, 1), (32, 2), (40, 2), (13, 11)])
@pytest.mark.parametrize("kind", ALL)
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_prefix_rows(D, kind, B, group):
    lens = [(7 * b) % 130 for b in range(B)]
    b = Batch(lens, 2 * group, 2, D, 16, "bf16" if D in (96, 256) else "fp16", kind, prefix=1003, seed=B + D)
    b.check(b.run(), rows=sorted({0, 1, B // 2, B - 2, B - 1}))


@pytest.mark.parametrize("prefix", [1, 31, 33, 2049])
@pytest.mark.parametrize("kind", ALL)
def test_prefix_lengths_many_rows(kind, prefix):
    b = Batch([3] * 70, 4, 2, 128, 32, "fp16", kind, prefix=prefix, seed=prefix)
    b.check(b.run(), rows=[0, 31, 69])


@pytest.mark.parametrize("kind", ["none", "int8"])
@pytest.mark.parametrize("B", [33, 52])
def test_prefix_of_more_tiles_than_a_look(B, kind):
    """32 key heads leave each part of the prefix more than 64 tiles."""
    b = Batch([5] * B, 32, 32, 64, 64, "fp16", kind, prefix=20011, seed=B)
    b.check(b.run(), rows=[0, B - 1])


@pytest.mark.parametrize("kind", ["int8", "fp4"])
def test_own_tokens_of_more_tiles_than_a_look(kind):
    """300 sequences of one long table row leave each wave more than 64 tiles."""
    import torch
    n, B = 25003, 300
    b = Batch([n], 2, 2, 64, 64, "fp16", kind, seed=1)
    b.table = b.table.repeat(B, 1)
    b.lens = [n - 100 * i for i in range(B)]
    b.lens[-2:] = [0, n]
    b.ld = dev(np.array(b.lens, np.int32))
    b.q = torch.from_numpy(np.random.default_rng(2).standard_normal((B, 2, 64)).astype(np.float32)).to(tdt("fp16")).cuda()
    b.check(b.run(), rows=[0, 1, 150, B - 2, B - 1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [16, 256, 257, 700])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128, 136, 256])
def test_adapter_ranks(R, M, dtype):
    c = Case(M, 1032, 203, R, 5, dtype, seed=M + R)
    c.check(c.run("residual"), "residual")


@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("N", [1, 3, 7, 8, 9, 63, 64, 71, 129, 1030])
def test_adapter_channels(N, M):
    for R in (16, 48, 200):
        c = Case(M, 136, N, R, 4, "fp16", seed=N + M)
        for epi in ("none", "gelu", "residual"):
            c.check(c.run(epi), epi)


@pytest.mark.parametrize("M,K", [(1, 40), (1, 5000), (20, 16376), (280, 8200), (280, 504), (1000, 3336), (9000, 72)])
def test_adapter_parts(M, K):
    c = Case(M, K, 40, 16, 3, "bf16", seed=K)
    c.check(c.run(), rows=slice(0, None) if M < 2000 else slice(M - 300, None))


def test_adapters_of_a_tile_all_different():
    """Sixteen adapters and none in each tile of rows, in the walk over many rows too."""
    for M in (32, 400):
        ids = np.arange(M) * 7 % 17 - 1
        c = Case(M, 128, 300, 24, 16, "fp16", seed=M, ids=ids)
        c.check(c.run("gelu"), "gelu")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("K", [8, 40, 1024, 1032, 2048, 2056])
@pytest.mark.parametrize("R", [8, 16, 24])
@pytest.mark.parametrize("M", [1, 2, 4, 5])
def test_adapters_of_few_rows(M, R, K, dtype):
    """On both sides of where one launch does for both products; a row's bits are the same beside others or alone."""
    import torch
    for ids in (None, [1, -1, 1, 0, 2][:M], [2] * M):
        c = Case(M, K, 75, R, 3, dtype, seed=M + K, ids=ids)
        out = c.run("residual")
        c.check(out, "residual")
        if ids is not None:
            first = c.run("residual", Y=c.Y[:1], X=c.X[:1], ids=c.ids[:1], residual=c.res[:1])
            assert torch.equal(first, out[:1])
            y = c.Y.clone()
            c.run(Y=y, out=y)
            c.check(y)


def calls():
    """One of each kind, in sizes that need a workspace."""
    from w4a4_post_quantized_zigzag_amd import binding as bd
    own = Batch([900, 17, 0, 2500], 8, 2, 128, 16, "bf16", "int8", seed=1)
    own4 = Batch([1200, 640, 33], 6, 2, 64, 32, "fp16", "fp4", seed=2)
    behind = Batch([5 * i for i in range(40)], 8, 2, 128, 16, "fp16", "none", prefix=3001, seed=3)
    few = Batch([9, 200], 4, 4, 64, 16, "bf16", "int8", prefix=700, seed=4)
    ad, rows = Case(40, 1032, 515, 24, 6, "fp16", seed=5), Case(600, 520, 130, 64, 3, "bf16", seed=6)
    size = lambda b, *n: (len(b.lens), b.H, b.KV, b.D, *n)  # noqa: E731
    L = bd.lib()
    return [(lambda ws: own.run(max_len=2500, ws=ws), L.w4a4_paged_attn_quant_workspace_bytes(*size(own, 2500, 0, 0))),
            (lambda ws: own4.run(max_len=1200, ws=ws), L.w4a4_paged_attn_quant_workspace_bytes(*size(own4, 1200, 0, 0))),
            (lambda ws: behind.run(max_prefix=3001, max_len=200, ws=ws),
             L.w4a4_paged_attn_shared_workspace_bytes(*size(behind, 3001, 200))),
            (lambda ws: few.run(max_prefix=700, max_len=200, ws=ws),
             L.w4a4_paged_attn_shared_workspace_bytes(*size(few, 700, 200))),
            (lambda ws: ad.run("gelu", ws=ws), L.w4a4_adapter_workspace_bytes(40, 1032, 24)),
            (lambda ws: rows.run("residual", ws=ws), L.w4a4_adapter_workspace_bytes(600, 520, 64))]


def test_calls_on_two_streams_at_once():
    import torch
    every = calls()
    buf = lambda n: torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")  # noqa: E731
    want = [f(buf(n)) for f, n in every]
    ws = [[buf(n) for _, n in every] for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                at = (turn + 2 * i) % len(every)       # another call beside it each time
                got[i].append((at, every[at][0](ws[i][at])))
    torch.cuda.synchronize()
    for some in got:
        for at, out in some:
            assert torch.equal(out, want[at]), at


def test_graphs_that_share_a_workspace():
    """Captured one by one with one workspace, replayed in any order, with eager calls between the replays."""
    import torch
    every = calls()
    ws = torch.full((max(n for _, n in every),), 0xFF, dtype=torch.uint8, device="cuda")
    want = [f(ws).clone() for f, _ in every]
    graphs, outs = [], []
    for f, _ in every:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f(ws))
        graphs.append(g)
    for turn in range(4):
        for at in (3 * turn + np.arange(len(every)) * (5 if turn % 2 else 1)) % len(every):
            outs[at].zero_()
            graphs[at].replay()
            assert torch.equal(outs[at], want[at]), (turn, at)
            assert torch.equal(every[(at + turn) % len(every)][0](ws), want[(at + turn) % len(every)])
        torch.cuda.synchronize()
