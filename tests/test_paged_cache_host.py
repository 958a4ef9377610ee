"""PagedCache.write and read over a 16-bit cache, whose rows are moved by indexing (no GPU needed): a slot outside the cache
is skipped and reads as zeros, as over a quantized one, and rows of another shape are refused."""
import pytest
import torch

from w4a4_post_quantized_zigzag_amd.stack import PagedCache

PAGES, HEADS, PAGE, D = 3, 2, 16, 64


@pytest.fixture
def cache():
    c = PagedCache.__new__(PagedCache)
    c.page_size, c.kind = PAGE, "fp16"
    c.kv = [tuple(torch.randn(PAGES, HEADS, PAGE, D).half() for _ in range(2))]
    return c


def rows(n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, HEADS, D, generator=g).half() for _ in range(2)]


END = PAGES * PAGE
SLOTS = [[5], [-1], [END - 1, 0, 16], [END, 3, -1, END + 7, 40], [3, -1, 2], [-1, -5, END], [-(1 << 62), 1 << 62, 17], [],
         [0, -1, 1], [END, 0]]


@pytest.mark.parametrize("slots", SLOTS)
def test_write_and_read(cache, slots):
    k, v = rows(len(slots))
    at = torch.tensor(slots, dtype=torch.int64)
    want = [t.clone() for t in cache.kv[0]]
    for w, x in zip(want, (k, v)):
        for s, row in zip(slots, x):
            if 0 <= s < END:
                w[s // PAGE, :, s % PAGE] = row
    cache.write(0, k, v, at)
    assert all(torch.equal(a, b) for a, b in zip(cache.kv[0], want))
    for got, x in zip(cache.read(0, at), (k, v)):
        keep = torch.tensor([0 <= s < END for s in slots], dtype=torch.bool).view(-1, 1, 1)
        assert torch.equal(got, x * keep)


def test_refusals(cache):
    k, v = rows(3)
    at = torch.tensor([1, 2, 3])
    before = [t.clone() for t in cache.kv[0]]
    for bad in ((k[:, :1], v), (k, v[:, :1]), (k[:2], v), (k[..., :1], v), (k[0], v[0])):
        with pytest.raises(ValueError, match="must be"):
            cache.write(0, *bad, at)
    for slots in (at[:2], at.view(1, 3)):
        with pytest.raises(ValueError, match="slots"):
            cache.write(0, k, v, slots)
    with pytest.raises(ValueError, match="slots"):
        cache.read(0, at.view(1, 3))
    assert all(torch.equal(a, b) for a, b in zip(cache.kv[0], before))
