"""How near kda_la_prefill's results have to be, as norms of the whole results:
the bounds, and the inputs that they are held on.

Final states, FP32.  The sums below are of independent roundings, so they add as
squares: exp of the decays behind a token, 2^-22 from the hardware's exponential
and as much from the sum that it is taken of (up to 2^3 in base 2, 8 additions);
its product with the key, 2^-24; 24 additions of the tensor cores a chunk, at
most 2^-23 each whichever way they round, sqrt(24) 2^-23 = 2^-20.7; earlier chunks
come in decayed to a tenth and less.  Together 2^-20.4: below 2^-20.  With keys of
two BF16 parts in place of three, each key would be short of its last bits by
2^-17 to 2^-16, all to one side: above 2^-20 (test_la_accuracy_host.py).

Outputs, BF16.  A rounding is off by 2^-8 / sqrt(3) of the power of two below a
value, 1.7e-3 of the values' norm.  There is the output's own, and in each of the
two sums of an output (the chunk's own tokens, the state before it) one of an
operand (the decayed scores, the state's copy): sqrt(2) 1.7e-3 = 2.4e-3."""

import torch

STATE_BOUND = 2.0 ** -20
OUT_BOUND = 3e-3
D = 128


def inputs(T, H, Hk, N, low, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = {"q": rnd(1, T, Hk, D).bfloat16(), "k": rnd(1, T, Hk, D).bfloat16(), "v": rnd(1, T, H, D).bfloat16(),
         "g": low * torch.rand((1, T, H), generator=gen)}
    return d, rnd(N, H, D, D)


# T, H, Hk, offsets of a packed batch, low: decays of 2.3 and 23 to a chunk.
CASES = [(300, 2, 1, None, -0.05), (1100, 3, 3, None, -0.05), (700, 2, 2, None, -0.5),
         (1300, 2, 1, [0, 300, 300, 1173, 1300], -0.05)]
