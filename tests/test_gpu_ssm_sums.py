"""kda_ssm_prefill's sums over the states, in FP32: outputs against the definition in
64 bits, with no part of the bound for a cut of the states or of C to fewer bits."""

import pytest
import torch

import ops_reference as ref
import scan_reference as scan
from test_gpu_ssm import BF16, F32, cuts, draw, kda, on_gpu, want_of  # noqa: F401

pytestmark = pytest.mark.gpu

# A sum of 64 products: a lane adds 8 of them in each of two halves and both halves, then
# four lanes' and two warps' sums are added: 12 roundings after the product's own, 13 2^-24 of
# the terms' magnitudes, below 2^-20, which scan_reference.py has already.
SUMS = 0.0


@pytest.mark.parametrize("S", [1, 5, 8, 16, 20, 32, 48, 64])
@pytest.mark.parametrize("dt,bc", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("gate", [True, False])
def test_sums(kda, S, dt, bc, gate):  # noqa: F811
    lead, dim, cu = (1, 200), 72, [0, 3, 90, 90, 200]
    for offsets in (None, cu):
        d = draw(lead, dim, S, S, G=2, dt=dt, bc=bc, z=gate, D=gate, init=1 if offsets is None else 4)
        o, f, oe, fe = want_of(d, offsets, cut=SUMS)
        on_dev = on_gpu(d)
        for on, chunks in ((False, 0), (True, 4)):
            kda.set_segments(on, chunks)
            out, fin = kda.ssm_prefill(**on_dev, cu_seqlens=None if offsets is None else torch.tensor(offsets, device="cuda"))
            ref.assert_close(out, o, oe + scan.rounded(o, BF16), "out")
            ref.assert_close(fin, f, fe, "final")


def test_no_bias(kda):  # noqa: F811
    """Terms of one sign: outputs, in BF16, are as often too large as too small.  Over 2^19 of
    them the mean of the roundings, each within 2^-8 of its output and evenly spread, is
    below 5 x 2^-8 / sqrt(3 x 2^19) < 1.6e-5; a step is within 2^-18 of itself."""
    T, dim = 512, 1024
    d = draw((1, T), dim, 16, 1, z=False, D=False)
    for key in ("x", "B", "C"):
        d[key] = d[key].abs()
    dev = on_gpu(d)
    out = kda.ssm_prefill(**dev)[0][0].double()
    A, s = dev["A"].double(), scan.steps(dev["dt"], dev["dt_bias"], True)[0]
    x, B, C = dev["x"][0].double(), dev["B"][0].double(), dev["C"][0].double()
    h = torch.zeros(dim, 16, dtype=torch.float64, device="cuda")
    y = torch.empty(T, dim, dtype=torch.float64, device="cuda")
    for t in range(T):
        h = torch.exp(s[t][:, None] * A) * h + (s[t] * x[t])[:, None] * B[t]
        y[t] = (h * C[t]).sum(-1)
    assert (out / y - 1).mean().abs() < 1.6e-5 + scan.STEP
