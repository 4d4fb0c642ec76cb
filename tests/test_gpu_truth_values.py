"""A flag whose truth value raises is refused before anything runs: no state is
advanced and no output written."""

import pytest
import torch

pytestmark = pytest.mark.gpu


class Unclear:
    def __bool__(self):
        raise ArithmeticError("neither true nor false")


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def bf(*s):
    return torch.ones(s, dtype=torch.bfloat16, device="cuda")


def f32(*s):
    return torch.ones(s, device="cuda")


def test_beta_is_logit(kda):
    state, out = f32(2, 3, 128, 128), bf(2, 3, 128)
    with pytest.raises(ArithmeticError):
        kda.kda_decode(bf(2, 3, 128), bf(2, 3, 128), bf(2, 3, 128), -f32(2, 3, 128), bf(2, 3), state, out=out,
                       beta_is_logit=Unclear())
    torch.cuda.synchronize()
    assert (state == 1).all() and (out == 1).all()


def test_gate_first(kda):
    out = 7 * bf(5, 128)
    with pytest.raises(ArithmeticError):
        kda.gated_norm(bf(5, 128), bf(128), bf(5, 128), gate_first=Unclear(), out=out)
    torch.cuda.synchronize()
    assert (out == 7).all()


def test_output_final_state(kda):
    state, out = f32(1, 2, 128, 128), 7 * bf(1, 9, 2, 128)
    with pytest.raises(ArithmeticError):
        kda.la_prefill(bf(1, 9, 2, 128), bf(1, 9, 2, 128), bf(1, 9, 2, 128), -f32(1, 9, 2), init_state=state, out=out,
                       output_final_state=Unclear())
    torch.cuda.synchronize()
    assert (state == 1).all() and (out == 7).all()
