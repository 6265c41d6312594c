"""CPU checks of calls of the block-scaled cache that are refused before anything is launched:
sizes past its limits, an input without its output."""
import pytest
import torch

from fp8_paged_kv_attn_gb300 import kvq
from test_block_refusals import INVALID, block_cache, call


@pytest.mark.parametrize("P", [16, 32, 64])
def test_attention_refuses_tables_whose_last_tile_passes_32_bits(P):
    """Token counters run past a length by up to two tiles of 128 tokens."""
    most = (2 ** 31 - 256) // P
    for n in (0, 4):
        assert call("attn", cache=block_cache(page_size=P), MP=most + 1, n=n) == INVALID
        assert call("attn", cache=block_cache(page_size=P), MP=(2 ** 31 - P) // P, n=n) == INVALID
    assert call("attn", cache=block_cache(page_size=P), MP=most, n=0) == 0


class Handle:
    """A cache's and a rope's stand-in: what the binding asks of them, on the host."""

    def __init__(self, *c):
        self._c = c

    def c(self):
        return self._c


def test_binding_refuses_an_input_or_output_alone(monkeypatch):
    monkeypatch.setattr(kvq, "_device", lambda t, name: -1)  # host tensors report device -1
    x, i = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32)
    cache, rope = Handle(None, -1, 2, 64), Handle(None, -1)
    for a, b in ((x, None), (None, x)):
        with pytest.raises(ValueError, match="missing"):
            kvq.kvq_rope_block_append(cache, rope, a, b, x, x, None, i, i[None])
        with pytest.raises(ValueError, match="missing"):
            kvq.kvq_rope(rope, i, x, x, a, b)
    with pytest.raises(ValueError, match="missing"):
        kvq.kvq_rope(rope, i, x, None)
