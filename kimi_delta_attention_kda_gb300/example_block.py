"""A small hybrid stack with the operators as a model uses them: blocks with
KDA and blocks with per-head-decay linear attention in turn, prompts as one
packed batch, then single tokens on a pool of states.

    python -m kimi_delta_attention_kda_gb300.example_block
    python -m kimi_delta_attention_kda_gb300.example_block --kinds kda+conv ssm la+conv ssm

runs every sequence twice: whole, and as a prompt whose last tokens come one by
one; and prints how far the two are apart.  The weights are random.  The
projections are torch matrix products; everything between them is this
library: ``kda_prefill`` or ``la_prefill`` (``kda_decode`` or ``la_decode``)
for the mixer, ``gated_norm`` after it, ``residual_norm`` between blocks; with
``+conv`` a short convolution (``conv_prefill``, ``conv_decode``) of q, k and v in
front of the mixer; and in blocks of the kind ``ssm`` the convolution and the
selective scan (``ssm_prefill``, ``ssm_decode``) for the mixer.
"""

from __future__ import annotations

import argparse
import math

import torch
import torch.nn.functional as F

import kimi_delta_attention_kda_gb300 as kda

D = kda.HEAD_DIM
KINDS = ("kda", "la", "kda", "la")


class Block:
    """One mixer with its projections: "kda" (a decay for each key channel, the
    delta rule) or "la" (a decay for each head, key heads shared by two), either with
    "+conv".  Its states, and their pools, are lists."""

    def __init__(self, kind, heads, gen):
        width = heads * D
        self.kind, _, conv = kind.partition("+")
        self.heads, self.conv, kind = heads, bool(conv), self.kind
        self.key_heads = heads // 2 if kind == "la" and heads % 2 == 0 else heads
        decays = heads if kind == "la" else width
        self.sizes = [self.key_heads * D, self.key_heads * D, width, width, decays] + ([heads] if kind == "kda" else [])

        def weight(*shape):
            return (torch.randn(shape, generator=gen) * shape[-1] ** -0.5).bfloat16().cuda()

        self.w_in, self.w_out = weight(sum(self.sizes), width), weight(width, width)
        self.norm, self.mix_norm, self.post_norm = (
            (1 + 0.1 * torch.randn(n, generator=gen)).bfloat16().cuda() for n in (width, D, width))
        if self.conv:
            self.filters = weight(sum(self.sizes[:3]), 4).split(self.sizes[:3])

    def project(self, y, convolve):
        """q, k, v and the output gate as heads, the log-decays, and beta's logits."""
        p = (y @ self.w_in.t()).split(self.sizes, dim=-1)
        # (q, k and v are read where they lie in the projection, and written as the mixer takes them.)
        done = [convolve(i, x) for i, x in enumerate(p[:3])] if self.conv else []
        p = done + [x.contiguous() for x in p[len(done):]]
        q, k = (x.view(-1, self.key_heads, D) for x in p[:2])
        v, z = (x.view(-1, self.heads, D) for x in p[2:4])
        if self.kind == "la":
            return q, k, v, z, -F.softplus(p[4].float()), None
        return q, k, v, z, (-5 * torch.sigmoid(p[4].float() - 3)).view(-1, self.heads, D), p[5]

    def finish(self, o, z):
        o = kda.gated_norm(o, self.mix_norm, z, activation="silu" if self.kind == "la" else "sigmoid")
        return o.view(o.shape[0], -1) @ self.w_out.t()

    def prompt(self, y, cu):
        """Packed tokens [T, width]; (what the block adds, the final states, the mixer's in FP32)."""
        states = []

        def convolve(i, x):
            x, state = kda.conv_prefill(x[None], self.filters[i], cu_seqlens=cu)
            states.append(state)
            return x[0]
        q, k, v, z, g, beta = self.project(y, convolve)
        one = [x[None] for x in (q, k, v, g)]
        if self.kind == "la":
            o, state = kda.la_prefill(*one, cu_seqlens=cu)
        else:
            o, state = kda.kda_prefill(*one, beta[None], cu_seqlens=cu, beta_is_logit=True)
        return self.finish(o[0], z), states + [state.float()]

    def token(self, y, pools, slots):
        """One token of each sequence [N, width], its states in its row of the pools."""
        q, k, v, z, g, beta = self.project(y, lambda i, x: kda.conv_decode(x, self.filters[i], pools[i], slots=slots))
        if self.kind == "la":
            o = kda.la_decode(q, k, v, g, pools[-1], slots)
        else:
            o = kda.kda_decode(q, k, v, g, beta, pools[-1], slots, beta_is_logit=True)
        return self.finish(o, z)


class ScanBlock:
    """The selective scan behind its convolution: a decay for each channel and
    state, step sizes, B and C from the convolved channels."""

    STATES = 16

    def __init__(self, heads, gen):
        width, S = heads * D, self.STATES
        self.width, self.rank = width, width // 16

        def weight(*shape):
            return (torch.randn(shape, generator=gen) * shape[-1] ** -0.5).bfloat16().cuda()

        self.w_in, self.w_out = weight(2 * width, width), weight(width, width)
        self.w_keys, self.w_dt, self.filter = weight(self.rank + 2 * S, width), weight(width, self.rank), weight(width, 4)
        self.norm, self.post_norm = ((1 + 0.1 * torch.randn(width, generator=gen)).bfloat16().cuda() for _ in range(2))
        self.A = -torch.arange(1, S + 1).float().repeat(width, 1).cuda()
        self.skip = torch.ones(width).cuda()
        step = torch.exp(math.log(1e-3) + math.log(100) * torch.rand(width, generator=gen))
        self.dt_bias = torch.log(torch.expm1(step)).cuda()

    def keys(self, x):
        """dt, B and C of convolved channels [rows, width]."""
        p = x @ self.w_keys.t()
        B, C = (y.unflatten(-1, (1, self.STATES)) for y in p[:, self.rank:].split(self.STATES, dim=-1))
        return p[:, :self.rank] @ self.w_dt.t(), B, C

    def prompt(self, y, cu):
        p = y @ self.w_in.t()
        x, conv_state = kda.conv_prefill(p[None, :, :self.width], self.filter, cu_seqlens=cu)
        dt, B, C = self.keys(x[0])
        o, state = kda.ssm_prefill(x, dt[None], self.A, B[None], C[None], self.skip, p[None, :, self.width:], self.dt_bias,
                                   cu_seqlens=cu)
        return o[0] @ self.w_out.t(), [conv_state, state]

    def token(self, y, pools, slots):
        p = y @ self.w_in.t()
        x = kda.conv_decode(p[:, :self.width], self.filter, pools[0], slots=slots)
        dt, B, C = self.keys(x)
        o = kda.ssm_decode(x, dt, self.A, B, C, pools[1], self.skip, p[:, self.width:], self.dt_bias, slots=slots)
        return o @ self.w_out.t()


class Stack:
    def __init__(self, kinds=KINDS, heads=4, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.width = heads * D
        self.blocks = [ScanBlock(heads, gen) if kind == "ssm" else Block(kind, heads, gen) for kind in kinds]
        self.last = torch.ones(self.width, dtype=torch.bfloat16, device="cuda")

    def run(self, x, mix):
        """x [rows, width] through the blocks; mix(i, y) is what block i adds."""
        after = [b.norm for b in self.blocks[1:]] + [self.last]
        y, r = kda.residual_norm(x, torch.zeros(x.shape, device=x.device), self.blocks[0].norm)
        for i, block in enumerate(self.blocks):
            y, r = kda.residual_norm(mix(i, y), r, after[i], post_weight=block.post_norm, residual_out=r)
        return y

    def prompt(self, x, cu):
        """(outputs [T, width], each block's states)."""
        states = []

        def mix(i, y):
            o, state = self.blocks[i].prompt(y, cu)
            states.append(state)
            return o
        return self.run(x, mix), states

    def token(self, x, pools, slots):
        return self.run(x, lambda i, y: self.blocks[i].token(y, pools[i], slots))


def compare(lengths=(300, 17, 1200, 64), tokens=16, heads=4, seed=0, kinds=KINDS):
    """The relative distance (Frobenius norm) between each sequence's last
    ``tokens`` outputs computed whole and token by token."""
    stack = Stack(kinds, heads, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    seqs = [torch.randn(n + tokens, stack.width, generator=gen).bfloat16().cuda() for n in lengths]

    def packed(parts):
        cu = torch.tensor([0] + [p.shape[0] for p in parts], device="cuda").cumsum(0)
        return torch.cat(parts), cu

    x, cu = packed(seqs)
    whole, _ = stack.prompt(x, cu)
    want = torch.stack([whole[e - tokens:e] for e in cu[1:].tolist()])

    _, states = stack.prompt(*packed([s[:-tokens] for s in seqs]))
    # The sequences' rows of the pool in another order than the batch, and
    # one padding row at the batch's end.
    n = len(lengths)
    slots = torch.tensor(list(range(n, 0, -1)) + [-1], dtype=torch.int32, device="cuda")
    pools = []
    for block in states:
        pools.append([])
        for s in block:
            pool = torch.zeros((n + 2,) + s.shape[1:], dtype=s.dtype, device="cuda")
            pool[slots[:n].long()] = s
            pools[-1].append(pool)
    got = []
    for t in range(tokens):
        now = torch.stack([s[s.shape[0] - tokens + t] for s in seqs] + [seqs[0][0]])
        got.append(stack.token(now, pools, slots)[:n])
    got = torch.stack(got, 1)
    if kda.device_status() != 0:
        raise RuntimeError("an operator reported an error")
    return ((got.double() - want.double()).norm() / want.double().norm()).item()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--lengths", type=int, nargs="+", default=[300, 17, 1200, 64])
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--heads", type=int, default=4)
    ap.add_argument("--kinds", nargs="+", default=list(KINDS), choices=["kda", "la", "kda+conv", "la+conv", "ssm"])
    a = ap.parse_args()
    print("%d sequences, the last %d tokens one by one: relative distance %.2e from the whole prompts"
          % (len(a.lengths), a.tokens, compare(a.lengths, a.tokens, a.heads, kinds=a.kinds)))


if __name__ == "__main__":
    main()
