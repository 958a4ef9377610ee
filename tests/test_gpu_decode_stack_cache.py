"""What a stack with attention refuses of a cache, before anything is written to it."""
import numpy as np
import pytest

from w4a4_post_quantized_zigzag_amd.stack import LINEARS, Attention, DeviceStack, PagedCache

from parity_util import dev
from test_gpu_decode_stack import weights

pytestmark = pytest.mark.gpu


def test_cache_with_fewer_layers():
    A = Attention(2, 1, 64)
    ds = DeviceStack(weights(A, 128, 256, 3, seed=1), 128, 1, w4g=LINEARS, group=64, attention=A)
    cache = PagedCache(2, A, 2, pages=2)
    cache.advance()
    X = dev(np.ones((2, 128), np.float16))
    with pytest.raises(ValueError, match="layers"):
        ds.run(X, 0, cache=cache)
    assert not any(t.any() for t in cache.k + cache.v)
    more = PagedCache(4, A, 2, pages=2)   # what is left of it is not touched
    more.advance()
    ds.run(X, 0, cache=more)
    assert more.k[2].any() and not more.k[3].any()
