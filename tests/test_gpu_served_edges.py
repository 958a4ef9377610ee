"""Edges of the serving calls that sizes and arguments allow. Oracle and tolerances as in the tests of each call."""
import pytest

from w4a4_post_quantized_zigzag_amd.stack import Attention, PagedCache

from test_gpu_kv_attn import Batch

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
