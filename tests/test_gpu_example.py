"""The example stack: prompts computed whole against prompts continued token by
token.

Bound: a block's BF16 values are rounded about five times in either way
(projections, mixer, norms), each rounding 1.5e-3 of a tensor's norm, and the
mixers' own errors are of that size; over four blocks, added up without
cancelling, 6e-2.  A lost state or a wrong slot gives a distance of order one.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,tokens,heads", [((300, 17, 1200, 64), 16, 4), ((1, 2), 3, 2), ((4000,), 4, 1)])
def test_example_block(lengths, tokens, heads):
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from kimi_delta_attention_kda_gb300 import example_block
    assert example_block.compare(lengths, tokens, heads) < 6e-2


def test_streams():
    """New outputs belong to the stream that the call runs on."""
    import kimi_delta_attention_kda_gb300 as kda
    rnd = lambda *s: torch.randn(s, device="cuda").bfloat16()  # noqa: E731
    q, k, v, x, w = rnd(1, 200, 2, 128), rnd(1, 200, 2, 128), rnd(1, 200, 2, 128), rnd(9, 128), rnd(128)
    g = -torch.rand(1, 200, 2, device="cuda")
    want = [*kda.la_prefill(q, k, v, g), kda.gated_norm(x, w, x), *kda.residual_norm(x, x, w)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        got = [*kda.la_prefill(q, k, v, g, stream=stream), kda.gated_norm(x, w, x, stream=stream),
               *kda.residual_norm(x, x, w, stream=stream)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # A block that the current stream still writes to is not handed out to another.
    big = torch.zeros(1 << 28, device="cuda")
    held = torch.empty_like(x)
    torch.cuda.synchronize()
    at = held.data_ptr()
    for _ in range(20):
        big.add_(1)
    held.zero_()
    del held
    out = kda.gated_norm(x, w, x, stream=side)
    torch.cuda.synchronize()
    assert out.data_ptr() != at and torch.equal(out, want[2])
