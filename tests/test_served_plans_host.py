"""How the attention behind a shared prefix is cut, seen through its workspace (no GPU): the parts of the prefix times the
blocks of 128 query rows of a key/value head are the workgroups that it gets, and one more sequence must not take most of
them away."""
import pytest

from w4a4_post_quantized_zigzag_amd import binding as bd


def prefix_parts(B, heads, kv_heads, D=64, prefix=65536):
    nbytes = bd.lib().w4a4_paged_attn_shared_workspace_bytes(B, heads, kv_heads, D, prefix, 1)
    return round(nbytes / (B * heads * (4 * D + 8))) - 1       # one part for the own token


@pytest.mark.parametrize("kv_heads", [1, 2, 4, 8])
@pytest.mark.parametrize("rows", [512, 1024, 2048, 4088, 4096, 4104, 4200, 8192, 8200, 12288, 16384, 16392, 32776, 65536])
def test_many_rows_keep_half_the_compute_units(rows, kv_heads):
    """From four to hundreds of blocks a key/value head: half of the 256 compute units at least."""
    parts, blocks = prefix_parts(rows // 8, 8 * kv_heads, kv_heads), -(-rows // 128)
    assert parts >= 1 and parts * blocks * kv_heads >= 128, (parts, blocks)


def test_no_more_parts_than_needed():
    """Rows enough for every compute unit take the prefix as a whole: a part is written and read again for each row."""
    assert prefix_parts(32768, 8, 1) == 1 and prefix_parts(1024, 256, 32) == 1
