"""kda_gated_norm's gate over the whole range in which its activation is not
zero in BF16.

Bounds: one rounding to BF16 (2^-8 of the value; 2^-134 where it is subnormal);
the sigmoid of z < 0 is exp(z), off by 2^-16 at -95, over 1 + exp(z), and an
FP32 number below 2^-126 from z = -87.3 on, whose rounding is 2^-150 / exp(-95) =
2^-12.9 of it at z = -95; sums over a row and all else stay below 2^-14."""

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("first", [False, True])
def test_gates_of_every_size(kda, act, first):
    z = torch.arange(-95.0, 95.25, 0.25).bfloat16()
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(z.numel(), D, generator=gen).bfloat16()
    w = 1 + 0.1 * torch.randn(D, generator=gen)
    for gate in (z[:, None].expand(-1, D).contiguous(),                     # a row of one size
                 z[torch.randint(0, z.numel(), x.shape, generator=gen)]):  # sizes mixed
        out = kda.gated_norm(x.cuda(), w.cuda(), gate.cuda(), activation=act, gate_first=first, eps=1e-6)
        want = ref.gated_norm(x, w, gate, act, first, 1e-6)
        ref.assert_close(out, want, (ref.HALF_BF16 + 2.0 ** -12) * want.abs() + 2.0 ** -133, "gated norm")
        if not first and act == "silu":
            at = (gate < -87.4) & (gate > -90)
            assert at.any() and (out.cpu()[at] != 0).all()
