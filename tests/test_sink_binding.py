"""Numbers that the binding of the attention with sinks and of reading back takes: refused before ctypes cuts them
to 32 bits (no GPU)."""
import pytest
import torch

import mixed_precision_quantized_kvq_b200 as kvq

LAY = kvq.Layout(128, 32, 8, window=16)


def args():
    z = lambda: torch.zeros(64, dtype=torch.uint8)  # noqa: E731
    c = kvq.PagedCache(z(), z(), z(), z(), z(), z(), torch.zeros((2, 4), dtype=torch.int32), 8)
    lens, cu = torch.ones(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    return c, torch.zeros((2, 32, 128), dtype=torch.bfloat16), lens, cu


@pytest.mark.parametrize("bad", [2 ** 31, 2 ** 32 + 5, 2 ** 40, 2 ** 63 - 1, -1, -2 ** 40])
@pytest.mark.parametrize("name", ["bound", "sinks", "span"])
def test_numbers_beyond_32_bits(name, bad):
    c, q, lens, cu = args()
    kw = dict(bound=8, sinks=4, span=64)
    kw[name] = bad
    what = {"bound": "max_(len|q|rows)"}.get(name, name)
    with pytest.raises(ValueError, match=what):
        kvq.sink_decode_attention(LAY, c, q, lens, kw["bound"], kw["sinks"], kw["span"])
    with pytest.raises(ValueError, match=what):
        kvq.sink_prefill_attention(LAY, c, q, cu, lens, kw["bound"], kw["sinks"], kw["span"])
    if name == "bound":
        with pytest.raises(ValueError, match=what):
            kvq.read_back(LAY, c, lens, cu, lens, 2, bad)


def test_the_largest_numbers_are_taken():
    c, q, lens, cu = args()
    with pytest.raises(ValueError, match="CUDA tensor"):     # the next check
        kvq.sink_decode_attention(LAY, c, q, lens, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)
