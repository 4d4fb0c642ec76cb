"""kda_la_prefill's results against the recurrence in 64 bits, as norms: the
final states to FP32 and the outputs to two BF16 roundings (la_accuracy.py has
the bounds and where they come from)."""

import pytest
import torch

import la_accuracy as la
import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


@pytest.mark.parametrize("seg", [0, 8, 24])
@pytest.mark.parametrize("T,H,Hk,cu,low", la.CASES)
def test_norms_of_the_errors(kda, T, H, Hk, cu, low, seg):
    d, init = la.inputs(T, H, Hk, len(cu) - 1 if cu else 1, low, T)
    dev = {key: x.cuda() for key, x in d.items()}
    kda.set_segments(True, seg)
    try:
        out, fin = kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], init_state=init.cuda(),
                                  cu_seqlens=None if cu is None else torch.tensor(cu, device="cuda"))
        torch.cuda.synchronize()
    finally:
        kda.set_segments(True, 0)
    assert kda.device_status() == 0
    o, f, _, _ = ref.la_tokens(d["q"], d["k"], d["v"], d["g"], init, cu)
    error = lambda got, want: ((got.cpu().double() - want).norm() / want.norm()).item()  # noqa: E731
    print("final state %.2e, out %.2e" % (error(fin, f), error(out, o)))
    assert error(fin, f) <= la.STATE_BOUND
    assert error(out, o) <= la.OUT_BOUND
