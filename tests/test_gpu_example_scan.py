"""The example stack with the short convolution and the selective scan in it: prompts
computed whole against prompts continued token by token.

Bound: as for the stack without them (6e-2 over four blocks), a block's values being
rounded to BF16 about five times in either way; with the convolution and the scan's projections
up to eight times, each 1.5e-3 of a tensor's norm, added up without cancelling over both
ways and four blocks: 4 * 2 * 8 * 1.5e-3 = 9.6e-2.  A lost state or a wrong slot gives a
distance of order one.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", [("kda+conv", "ssm", "la+conv", "ssm"), ("ssm",)])
@pytest.mark.parametrize("lengths,tokens,heads", [((300, 17, 1200, 64), 16, 4), ((1, 2), 3, 2), ((4000,), 4, 1)])
def test_example_block(kinds, lengths, tokens, heads):
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kimi_delta_attention_kda_gb300 import example_block
    assert example_block.compare(lengths, tokens, heads, kinds=kinds) < 9.6e-2
