"""The short causal convolution and the selective scan from their definitions,
in 64 bits on the CPU, with what the tests' error bounds are made of."""

import torch

from ops_reference import HALF_BF16


def silu(x):
    return x * torch.sigmoid(x)


def ranges(x, cu):
    """(row of the batch, first token, end) of each sequence."""
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    return [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]


def conv(x, w, bias=None, init=None, cu=None, act="silu"):
    """(out, final, bound on the FP32 work's error in out).

    y is a sum of W + 1 terms, each step off by 2^-24 of the terms' magnitudes at
    most: 2^-21 of their sum for W up to 4.  silu' is within 1.1, and the sigmoid is off by
    2^-21 + 2^-24 |y| of itself.
    """
    x, w = x.double(), w.double()
    W = w.shape[1]
    out, mag = torch.zeros_like(x), torch.zeros_like(x)
    finals = []
    for n, (b, lo, hi) in enumerate(ranges(x, cu)):
        head = torch.zeros(W - 1, x.shape[2], dtype=torch.float64) if init is None else init[n].double()
        rows = torch.cat([head, x[b, lo:hi]])
        for t in range(hi - lo):
            y = (rows[t:t + W] * w.t()).sum(0)
            m = (rows[t:t + W] * w.t()).abs().sum(0)
            if bias is not None:
                y, m = y + bias.double(), m + bias.double().abs()
            out[b, lo + t] = silu(y) if act == "silu" else y
            mag[b, lo + t] = 1.1 * 2.0 ** -21 * m + (2.0 ** -20 + 2.0 ** -23 * y.abs()) * y.abs()
        finals.append(rows[hi - lo:])
    return out, torch.stack(finals), mag


def steps(dt, bias, softplus):
    u = dt.double()
    if bias is not None:
        u = u + bias.double()
    return torch.logaddexp(u, torch.zeros_like(u)) if softplus else u


# One step's relative error in FP32.  dt: its sum with the bias 2^-24 of |u| + |bias|,
# the exponential's argument 2^-23 |u| and itself 1.4e-7, the logarithm 1.8e-7: for
# |u| and |bias| up to 16, 16 2^-24 + 16 2^-23 + 2^-21.5 < 2^-18.  A decay exp(dt A):
# |dt A| 2^-18 + 2^-22, and x exp(-x) is below 0.37; an addend, one more product or two.
STEP = 2.0 ** -18


def scan(x, dt, A, B, C, D=None, z=None, bias=None, softplus=True, init=None, cu=None, cut=2.0 ** -10 + 2.0 ** -11):
    """(out, final, out's bound but for its own rounding, final's bound likewise).

    E is the error of the states if every step's decay and addend are off by a part of
    themselves: E <- a E + a |h| + |b|, in units of STEP; what a cut into spans adds (a decay from
    a sum of dt, one more product for each span) is of the kind and less than one
    more step for each, so everything is doubled.  `cut` is the part of |C h| that
    rounding h and C on the way to out may cost: TF32, 10 bits kept, h cut off (2^-10) and
    C rounded (2^-11).
    """
    x, A, B, C = x.double(), A.double(), B.double(), C.double()
    s = steps(dt, bias, softplus)
    per = x.shape[-1] // B.shape[-2]
    B, C = B.repeat_interleave(per, -2), C.repeat_interleave(per, -2)
    gate = silu(z.double()) if z is not None else torch.ones_like(x)
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    finals, bounds = [], []
    for n, (b, lo, hi) in enumerate(ranges(x, cu)):
        h = torch.zeros_like(A) if init is None else init[n].double()
        mag, E = h.abs(), torch.zeros_like(A)
        for t in range(lo, hi):
            a = torch.exp(s[b, t][:, None] * A)
            add = (s[b, t] * x[b, t])[:, None] * B[b, t]
            E = a * E + a * mag + add.abs()
            h, mag = a * h + add, a * mag + add.abs()
            y = (C[b, t] * h).sum(-1)
            off = 2 * STEP * (C[b, t].abs() * E).sum(-1) + (cut + 2.0 ** -20) * (C[b, t] * h).abs().sum(-1)
            if D is not None:
                skip = D.double() * x[b, t]
                y, off = y + skip, off + 2.0 ** -22 * (skip.abs() + y.abs())
            out[b, t] = y * gate[b, t]
            bound[b, t] = off * gate[b, t].abs() + 2.0 ** -19 * out[b, t].abs()
        finals.append(h)
        bounds.append(2 * STEP * E)
    return out, torch.stack(finals), bound, torch.stack(bounds)


def rounded(want, dtype):
    """What rounding `want` to the type may add."""
    return HALF_BF16 * want.abs() if dtype == torch.bfloat16 else torch.zeros_like(want)
