"""A small hybrid stack with the operators as a model uses them: blocks with
KDA and blocks with per-head-decay linear attention in turn, prompts as one
packed batch, then single tokens on a pool of states.

    python -m kimi_delta_attention_kda_gb300.example_block

runs every sequence twice: whole, and as a prompt whose last tokens come one by
one; and prints how far the two are apart.  The weights are random.  The
projections are torch matrix products; everything between them is this
library: ``kda_prefill`` or ``la_prefill`` (``kda_decode`` or ``la_decode``)
for the mixer, ``gated_norm`` after it, ``residual_norm`` between blocks.
"""

from __future__ import annotations

import argparse

import torch
import torch.nn.functional as F

import kimi_delta_attention_kda_gb300 as kda

D = kda.HEAD_DIM


class Block:
    """One mixer with its projections: "kda" (a decay for each key channel, the
    delta rule) or "la" (a decay for each head, key heads shared by two)."""

    def __init__(self, kind, heads, gen):
        width = heads * D
        self.kind, self.heads = kind, heads
        self.key_heads = heads // 2 if kind == "la" and heads % 2 == 0 else heads
        decays = heads if kind == "la" else width
        self.sizes = [self.key_heads * D, self.key_heads * D, width, width, decays] + ([heads] if kind == "kda" else [])

        def weight(*shape):
            return (torch.randn(shape, generator=gen) * shape[-1] ** -0.5).bfloat16().cuda()

        self.w_in, self.w_out = weight(sum(self.sizes), width), weight(width, width)
        self.norm, self.mix_norm, self.post_norm = (
            (1 + 0.1 * torch.randn(n, generator=gen)).bfloat16().cuda() for n in (width, D, width))

    def project(self, y):
        """q, k, v and the output gate as heads, the log-decays, and beta's logits."""
        p = [x.contiguous() for x in (y @ self.w_in.t()).split(self.sizes, dim=-1)]
        q, k = (x.view(-1, self.key_heads, D) for x in p[:2])
        v, z = (x.view(-1, self.heads, D) for x in p[2:4])
        if self.kind == "la":
            return q, k, v, z, -F.softplus(p[4].float()), None
        return q, k, v, z, (-5 * torch.sigmoid(p[4].float() - 3)).view(-1, self.heads, D), p[5]

    def finish(self, o, z):
        o = kda.gated_norm(o, self.mix_norm, z, activation="silu" if self.kind == "la" else "sigmoid")
        return o.view(o.shape[0], -1) @ self.w_out.t()

    def prompt(self, y, cu):
        """Packed tokens [T, width]; (what the block adds, the final states in FP32)."""
        q, k, v, z, g, beta = self.project(y)
        one = [x[None] for x in (q, k, v, g)]
        if self.kind == "la":
            o, state = kda.la_prefill(*one, cu_seqlens=cu)
        else:
            o, state = kda.kda_prefill(*one, beta[None], cu_seqlens=cu, beta_is_logit=True)
        return self.finish(o[0], z), state.float()

    def token(self, y, pool, slots):
        """One token of each sequence [N, width], its state in its row of the pool."""
        q, k, v, z, g, beta = self.project(y)
        if self.kind == "la":
            o = kda.la_decode(q, k, v, g, pool, slots)
        else:
            o = kda.kda_decode(q, k, v, g, beta, pool, slots, beta_is_logit=True)
        return self.finish(o, z)


class Stack:
    def __init__(self, kinds=("kda", "la", "kda", "la"), heads=4, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.width = heads * D
        self.blocks = [Block(kind, heads, gen) for kind in kinds]
        self.last = torch.ones(self.width, dtype=torch.bfloat16, device="cuda")

    def run(self, x, mix):
        """x [rows, width] through the blocks; mix(i, y) is what block i adds."""
        after = [b.norm for b in self.blocks[1:]] + [self.last]
        y, r = kda.residual_norm(x, torch.zeros(x.shape, device=x.device), self.blocks[0].norm)
        for i, block in enumerate(self.blocks):
            y, r = kda.residual_norm(mix(i, y), r, after[i], post_weight=block.post_norm, residual_out=r)
        return y

    def prompt(self, x, cu):
        """(outputs [T, width], each block's states [N, heads, 128, 128])."""
        states = []

        def mix(i, y):
            o, state = self.blocks[i].prompt(y, cu)
            states.append(state)
            return o
        return self.run(x, mix), states

    def token(self, x, pools, slots):
        return self.run(x, lambda i, y: self.blocks[i].token(y, pools[i], slots))


def compare(lengths=(300, 17, 1200, 64), tokens=16, heads=4, seed=0):
    """The relative distance (Frobenius norm) between each sequence's last
    ``tokens`` outputs computed whole and token by token."""
    stack = Stack(heads=heads, seed=seed)
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
    for s in states:
        pool = torch.zeros((n + 2,) + s.shape[1:], device="cuda")
        pool[slots[:n].long()] = s
        pools.append(pool)
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
    a = ap.parse_args()
    print("%d sequences, the last %d tokens one by one: relative distance %.2e from the whole prompts"
          % (len(a.lengths), a.tokens, compare(a.lengths, a.tokens, a.heads)))


if __name__ == "__main__":
    main()
