"""The example of a served attention block (examples/attention_block.py) runs its prompt and single-token
steps, and its outputs are as near to the unquantized block as its quantizers allow."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (4, 4)])
def test_block_of_a_served_model(heads, kv_heads):
    """MXFP4's relative error of normal values is about 0.12 (codes 1 to 3 bits of significand, power-of-two
    scales) and enters four times: x and the fused weight, o and the output weight, each product carrying
    the root of the sum of its operands' squares (0.17); the values' 0.17 is averaged over the keys like the
    values themselves, so the two products together carry 0.24. E4M3's 0.03 and the scores' error add
    little. Bound: twice that."""
    import attention_block
    prompt, single = attention_block.run(hidden=1024, heads=heads, kv_heads=kv_heads, tokens=150, steps=4)
    assert 0.0 < prompt < 0.48 and 0.0 < single < 0.48
