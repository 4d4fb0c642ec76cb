"""The bound on kda_la_prefill's final states tells three BF16 parts of a key
from two: the recurrence in 64 bits with the decayed keys of each chunk of 128
tokens cut by truncation as the kernel cuts them (no GPU needed)."""

import pytest
import torch

import la_accuracy as la
import ops_reference as ref

CHUNK = 128


def truncated(x):
    """The upper half of each FP32 word."""
    return (x.view(torch.int32) & -65536).view(torch.float32)


def final_states(d, init, cu, parts):
    q, k, v, g = (d[x][0] for x in ("q", "k", "v", "g"))
    T, H = v.shape[:2]
    k = k.repeat_interleave(H // k.shape[1], 1)
    states = []
    for n, (lo, hi) in enumerate(zip(cu, cu[1:])):
        S = init[n].double()
        for at in range(lo, hi, CHUNK):
            s = slice(at, min(at + CHUNK, hi))
            G = g[s].double()
            behind = G.flip(0).cumsum(0).flip(0) - G
            key = k[s].float() * behind.exp().float()[..., None]
            left, total = key, torch.zeros_like(key, dtype=torch.float64)
            for _ in range(parts):
                part = truncated(left)
                total += part.double()
                left = left - part
            S = S * G.sum(0).exp()[:, None, None] + torch.einsum("thv,thk->hvk", v[s].double(), total)
        states.append(S)
    return torch.stack(states)


@pytest.mark.parametrize("T,H,Hk,cu,low", la.CASES)
def test_two_parts_are_not_enough(T, H, Hk, cu, low):
    d, init = la.inputs(T, H, Hk, len(cu) - 1 if cu else 1, low, T)
    f = ref.la_tokens(d["q"], d["k"], d["v"], d["g"], init, cu)[1]
    error = lambda parts: ((final_states(d, init, cu or [0, T], parts) - f).norm() / f.norm()).item()  # noqa: E731
    assert error(3) < la.STATE_BOUND / 4       # the roundings of a product and of exp alone
    assert error(2) > 1.5 * la.STATE_BOUND
    assert error(1) > 100 * la.STATE_BOUND
