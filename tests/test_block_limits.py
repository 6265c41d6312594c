"""CPU checks of the limits of the block-scaled cache's sizes: calls that are refused before
anything is launched."""
import pytest

from test_block_refusals import INVALID, block_cache, call


@pytest.mark.parametrize("P", [16, 32, 64])
def test_attention_refuses_tables_whose_last_tile_passes_32_bits(P):
    """Token counters run past a length by up to two tiles of 128 tokens."""
    most = (2 ** 31 - 256) // P
    for n in (0, 4):
        assert call("attn", cache=block_cache(page_size=P), MP=most + 1, n=n) == INVALID
        assert call("attn", cache=block_cache(page_size=P), MP=(2 ** 31 - P) // P, n=n) == INVALID
    assert call("attn", cache=block_cache(page_size=P), MP=most, n=0) == 0
