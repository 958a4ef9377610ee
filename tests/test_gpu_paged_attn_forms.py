"""The forms that the one-token attention takes over long sequences, for every head size: one wave per split and
four, few splits and the most, more splits than the join loads ahead, a length hint that is far above or below
the lengths (a captured call passes what its cache can hold) and windows that hide nothing. Tolerances are
those derived in test_gpu_paged_attn."""
import numpy as np
import pytest

from w4a4_post_quantized_zigzag_amd import binding as bd

from test_gpu_paged_attn import Batch

pytestmark = pytest.mark.gpu

DIMS = [64, 96, 128, 192, 256]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("H,KV", [(8, 1), (6, 3), (20, 1)])
def test_split_and_joined(H, KV, D, dtype):
    """1001 tokens: one tile per one-wave workgroup; hints above it leave whole runs to few of them."""
    b = Batch([1001], H, KV, D, 16, dtype, seed=H + D)
    for max_len in (1001, 300, 9000, 1 << 17, 1 << 30):
        b.check(b.run(max_len=max_len))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
def test_most_splits(D, dtype):
    """One wave on a tile in as many workgroups as one sequence gets, four waves in as many as there are splits,
    beyond what the join loads ahead; and hints below the length, whose last split takes what is left."""
    b = Batch([3050], 2, 1, D, 32, dtype, seed=D)
    for max_len in (3050, 2900):
        b.check(b.run(max_len=max_len))
    b = Batch([33001], 2, 1, D, 32, dtype, seed=D + 1)
    for max_len in (33001, 30000, 8192, 1 << 20):
        b.check(b.run(max_len=max_len))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
def test_ragged_lengths_under_a_loose_hint(D, dtype):
    """Every row takes its own path through one plan: nothing, one tile, one split, several."""
    lens = [2500, 0, 1, 33, 640, 128, 1999, 4097]
    b = Batch(lens, 4, 2, D, 64, dtype, seed=D)
    for max_len in (None, 4097, 100, 1 << 14, 1 << 17):
        b.check(b.run(max_len=max_len))


@pytest.mark.parametrize("window,sinks", [(4097, 0), (5000, 3), (4090, 70), (1 << 20, 1 << 20), ((1 << 31) - 1, (1 << 31) - 1)])
def test_a_window_that_hides_nothing(window, sinks):
    """The same tokens are visible as without one."""
    b = Batch([4097, 0, 700, 64, 1, 3000], 8, 2, 128, 16, "bf16", seed=5)
    b.check(b.run(window=window, sinks=sinks))


@pytest.mark.parametrize("max_len", [None, 700, 1 << 17])
@pytest.mark.parametrize("window,sinks", [(300, 0), (300, 40), (1000, 4), (2047, 33)])
def test_windows_over_split_sequences(window, sinks, max_len):
    b = Batch([5003, 10, 1004, 299, 341, 2500], 6, 1, 96, 16, "fp16", seed=window)
    b.check(b.run(window=window, sinks=sinks, max_len=max_len), window=window, sinks=sinks)


def test_captured_with_the_capacity_of_the_cache():
    """One graph, captured with the capacity as its hint, serves lengths from nothing to thousands."""
    import torch
    b = Batch([6000, 2, 800], 8, 2, 128, 16, "bf16", seed=7)
    full = list(b.lens)
    out = torch.empty_like(b.q)
    b.run(max_len=1 << 16, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(max_len=1 << 16, out=out)
    rng = np.random.default_rng(0)
    for turn in range(5):
        b.lens = [int(rng.integers(0, n + 1)) for n in full] if turn else full
        b.ld.copy_(torch.tensor(b.lens, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, b.run(max_len=1 << 16)), turn
        b.check(got)
        torch.cuda.synchronize()


@pytest.mark.parametrize("D", DIMS)
def test_bad_pages_and_lengths_in_split_sequences(D):
    """A page entry that names no page, in any split, and a length beyond the table make their sequence NaN."""
    import torch
    b = Batch([4000, 4000, 4000, 4000, 4000], 2, 1, D, 16, "fp16", seed=D)
    b.table[0, 0], b.table[1, 249], b.table[2, 120] = -1, b.P, 1 << 30
    b.ld[3] = b.table.shape[1] * 16 + 1
    for max_len in (4000, 32, 1 << 17):
        out = b.run(max_len=max_len)
        assert bool(torch.isnan(out[:4]).all()), max_len
        b.check(out, rows=[4])


def test_workspace_covers_every_hint():
    """The size query is for the call's own hint: a workspace of just that size is accepted, one byte less not."""
    import torch
    b = Batch([3000, 17], 8, 2, 192, 16, "fp16", seed=3)
    for max_len in (1, 400, 3000, 40000, 1 << 20):
        need = bd.lib().w4a4_paged_attn_workspace_bytes(2, 8, 2, 192, max_len, 0, 0)
        ws = torch.full((max(need, 256) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        out = b.run(max_len=max_len, ws=ws[:max(need, 256)])
        assert bool((ws[max(need, 256):] == 0xFF).all())
        b.check(out)
        if need:
            with pytest.raises(bd.W4A4Error, match="workspace"):
                b.run(max_len=max_len, ws=ws[:need - 1])
