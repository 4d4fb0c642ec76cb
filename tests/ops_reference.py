"""The operators around the prefill from their definitions, in 64 bits on the
CPU, with the magnitudes that the tests' error bounds are made of.

Each function returns its results and, for every result, the same sums taken
over absolute values: a rounding of any operand by a relative amount r moves a
result by at most r times that magnitude.
"""

import torch

D = 128
SCALE = D ** -0.5

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2     # 2^-8
HALF_F32 = torch.finfo(torch.float32).eps / 2       # 2^-24


def la_tokens(q, k, v, g, init=None, cu=None, scale=SCALE):
    """Token by token: (out, final, |out|, |final|); packed with cu (a list)."""
    q, k, v, g = (x.double() for x in (q, k, v, g))
    B, T, H, _ = v.shape
    rep = H // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    if g.dim() == 1:
        g = g.expand(B, T, H)
    ranges = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    out, mag = torch.zeros_like(v), torch.zeros_like(v)
    finals, mags = [], []
    for n, (b, lo, hi) in enumerate(ranges):
        S = torch.zeros(H, D, D, dtype=torch.float64) if init is None else init[n].double().clone()
        A = S.abs()
        for t in range(lo, hi):
            e = g[b, t].exp()[:, None, None]
            vk = v[b, t][:, :, None] * k[b, t][:, None, :]
            # exp(-inf) S is 0 for every finite S.
            S = S * e + vk
            A = A * e + vk.abs()
            out[b, t] = scale * (S @ q[b, t][:, :, None])[..., 0]
            mag[b, t] = abs(scale) * (A @ q[b, t].abs()[:, :, None])[..., 0]
        finals.append(S)
        mags.append(A)
    return out, torch.stack(finals), mag, torch.stack(mags)


def la_step(q, k, v, g, S, scale=SCALE):
    """(out, state, |out|, |state|) of one token for states S [N, H, 128, 128]."""
    q, k, v, g, S = (x.double() for x in (q, k, v, g, S))
    rep = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    e = g.exp().expand(v.shape[:2])[..., None, None]
    vk = v[..., :, None] * k[..., None, :]
    new, mag = S * e + vk, S.abs() * e + vk.abs()
    return (scale * (new * q[..., None, :]).sum(-1), new,
            abs(scale) * (mag * q.abs()[..., None, :]).sum(-1), mag)


def kda_step(q, k, v, g, beta, S, logit=False):
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    if logit:
        beta = torch.sigmoid(beta)
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    e = g.exp()[..., None, :]
    S = S * e
    A = S.abs()
    u = beta[..., None] * (v - (S * k[..., None, :]).sum(-1))
    ua = beta[..., None] * (v.abs() + (A * k.abs()[..., None, :]).sum(-1))
    new = S + u[..., :, None] * k[..., None, :]
    mag = A + ua[..., :, None] * k.abs()[..., None, :]
    return (SCALE * (new * q[..., None, :]).sum(-1), new,
            SCALE * (mag * q.abs()[..., None, :]).sum(-1), mag)


def act(z, name):
    if name == "none" or z is None:
        return 1.0
    z = z.double()
    return torch.sigmoid(z) if name == "sigmoid" else z * torch.sigmoid(z)


def gated_norm(x, w, gate, name, first, eps):
    x, w, a = x.double(), w.double(), act(gate, name)
    if first:
        x = x * a
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return y if first else y * a


def residual_norm(x, r, w, post, gate, scale, eps):
    """(out, residual, |residual|)."""
    u = x.double()
    if post is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * post.double()
    if gate is not None:
        u = u * gate.double()
    new = r.double() + scale * u
    out = new / torch.sqrt((new * new).mean(-1, keepdim=True) + eps) * w.double()
    return out, new, r.double().abs() + abs(scale) * u.abs()


def assert_close(got, want, bound, what):
    """Every value within `bound` of `want`; NaN and infinities in the same places."""
    got, want = got.double().cpu(), want.double()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), "%s: values that are not finite in other places" % what
    err = torch.where(fine, (got - want).abs(), torch.zeros_like(want))
    bound = torch.where(fine, bound.expand_as(want), torch.zeros_like(want))
    over = err > bound
    if over.any():
        at = (err - bound).argmax()
        raise AssertionError("%s: %d of %d values over their bound; worst: %.6g for %.6g, bound %.3g" % (
            what, int(over.sum()), over.numel(), got.flatten()[at], want.flatten()[at], bound.flatten()[at]))
