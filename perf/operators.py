"""Cases for measuring the operators around the KDA prefill: linear attention
with a decay for each head (whole prompts and single tokens), the KDA step for
single tokens, and the norms around a block.

``run`` computes an operator in its plain form (torch, 32 bits) or, with
``own``, through this package; ``exact`` gives the definition in 64 bits.
"""

import math

import torch

own = False

DIM = 128
SCALE = 1.0 / math.sqrt(DIM)
EPS = 1e-6
CHUNK = 64                      # tokens per chunk of the plain chunked form
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HEADS = (1, 2, 3, 5, 6, 8, 12, 16, 32, 48, 64, 96)


def listed():
    return [
        # A prompt of the default benchmark's length on a small tensor-parallel
        # shard, going on from a state.
        {"name": "la_prefill t8192 h6", "op": "la_prefill", "B": 1, "T": 8192, "H": 6, "Hk": 6, "packed": False,
         "g": "token", "state": "fp32", "init": True},
        # The same prompt at the full head count.
        {"name": "la_prefill t8192 h96", "op": "la_prefill", "B": 1, "T": 8192, "H": 96, "Hk": 96, "packed": False,
         "g": "token", "state": "fp32", "init": False},
        # A packed batch of ragged prompts, three value heads to a key head.
        {"name": "la_prefill packed8 h12", "op": "la_prefill", "B": 8, "T": 33333, "H": 12, "Hk": 4, "packed": True,
         "g": "token", "state": "bf16", "init": True},
        # Short prompts with a constant decay for each head: latency.
        {"name": "la_prefill b3 t77 h6", "op": "la_prefill", "B": 3, "T": 77, "H": 6, "Hk": 6, "packed": False,
         "g": "head", "state": "fp32", "init": False},
        # One conversation on a shard: the latency of a token.
        {"name": "la_decode n1 h6", "op": "la_decode", "N": 1, "H": 6, "Hk": 6, "pool": 4, "pad": 0,
         "g": "token", "state": "fp32"},
        # A serving batch padded to a captured graph's size.
        {"name": "la_decode n128 h96", "op": "la_decode", "N": 128, "H": 96, "Hk": 32, "pool": 130, "pad": 3,
         "g": "token", "state": "bf16"},
        {"name": "kda_decode n1 h6", "op": "kda_decode", "N": 1, "H": 6, "pool": 4, "pad": 0, "state": "bf16",
         "logit": False},
        {"name": "kda_decode n64 h96", "op": "kda_decode", "N": 64, "H": 96, "pool": 67, "pad": 1, "state": "fp32",
         "logit": True},
        # After the mixer: a decode batch on a shard, and a whole prompt.
        {"name": "gated_norm m7 h6", "op": "gated_norm", "M": 7, "H": 6, "act": "sigmoid", "first": False,
         "weight": "bf16"},
        {"name": "gated_norm m8192 h96", "op": "gated_norm", "M": 8192, "H": 96, "act": "silu", "first": True,
         "weight": "fp32"},
        # Between two blocks: one token, and a whole prompt at 96 heads' width.
        {"name": "residual_norm m1 d768", "op": "residual_norm", "M": 1, "D": 768, "post": False, "gate": False,
         "scale": 1.0, "residual": "bf16", "weight": "bf16"},
        {"name": "residual_norm m8192 d12288", "op": "residual_norm", "M": 8192, "D": 12288, "post": True,
         "gate": True, "scale": 0.5, "residual": "fp32", "weight": "fp32"},
    ]


def _log(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n - 1 if n % 1024 == 0 else n


def draw(rng):
    op = rng.choice(("la_prefill", "la_prefill", "la_decode", "kda_decode", "gated_norm", "residual_norm"))
    H = rng.choice(HEADS)
    Hk = rng.choice([x for x in range(1, H + 1) if H % x == 0])
    if op == "la_prefill":
        T = _log(rng, 1, min(65536, 8192 * 96 // H))
        B = _log(rng, 1, max(1, min(32, 8192 * 96 // (H * T))))
        packed = rng.random() < 0.5
        return {"op": op, "B": B, "T": B * T if packed else T, "H": H, "Hk": Hk, "packed": packed,
                "g": rng.choice(("token", "token", "head")), "state": rng.choice(("fp32", "bf16")),
                "init": rng.random() < 0.5}
    if op == "la_decode":
        state = rng.choice(("fp32", "bf16"))
        N = _log(rng, 1, min(1024, 128 * 96 // H // (2 if state == "fp32" else 1)))
        return {"op": op, "N": N, "H": H, "Hk": Hk, "pool": N + rng.randint(0, 5), "pad": min(N - 1, rng.randint(0, 3)),
                "g": rng.choice(("token", "token", "head")), "state": state}
    if op == "kda_decode":
        N = _log(rng, 1, min(1024, 64 * 96 // H))
        return {"op": op, "N": N, "H": H, "pool": N + rng.randint(0, 5), "pad": min(N - 1, rng.randint(0, 3)),
                "state": rng.choice(("fp32", "bf16")), "logit": rng.random() < 0.5}
    if op == "gated_norm":
        return {"op": op, "M": _log(rng, 1, 8192 * 96 // H), "H": H, "act": rng.choice(("sigmoid", "silu", "none")),
                "first": rng.random() < 0.5, "weight": rng.choice(("fp32", "bf16"))}
    D = DIM * H if rng.random() < 0.7 else _log(rng, 1, 12288)
    return {"op": op, "M": _log(rng, 1, min(65536, 8192 * 12288 // D)), "D": D, "post": rng.random() < 0.5,
            "gate": rng.random() < 0.5, "scale": rng.choice((1.0, 0.5, 1.4142)),
            "residual": rng.choice(("fp32", "bf16")), "weight": rng.choice(("fp32", "bf16"))}


def _lengths(case, seed):
    """Ragged lengths of a packed batch, whole numbers that add up to T."""
    B, T = case["B"], case["T"]
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, T + 1, (B - 1,), generator=gen).sort().values.tolist()
    ends = [0] + cuts + [T]
    return [ends[i + 1] - ends[i] for i in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (std * torch.randn(shape, generator=gen, device=dev)).to(dtype)

    def decay(*shape):
        # Step sizes softplus(N(0, 1)) times rates that are spread over the
        # heads from 1/64 to 1.
        rate = torch.exp2(6 * torch.rand(shape[-1], generator=gen, device=dev) - 6)
        return -rate * torch.nn.functional.softplus(torch.randn(shape, generator=gen, device=dev))

    s = {"case": dict(case)}
    op = case["op"]
    if op == "la_prefill":
        B, T, H, Hk = (case[x] for x in ("B", "T", "H", "Hk"))
        lead = (1, T) if case["packed"] else (B, T)
        s["q"], s["k"], s["v"] = normal(*lead, Hk, DIM), normal(*lead, Hk, DIM), normal(*lead, H, DIM)
        s["g"] = decay(*lead, H) if case["g"] == "token" else decay(H)
        s["init"] = normal(B, H, DIM, DIM, dtype=DTYPES[case["state"]]) if case["init"] else None
        if case["packed"]:
            s["lengths"] = _lengths(case, seed)
            s["cu"] = torch.tensor([0] + s["lengths"], device=dev).cumsum(0)
    elif op in ("la_decode", "kda_decode"):
        N, H, P, pad = (case[x] for x in ("N", "H", "pool", "pad"))
        Hk = case.get("Hk", H)
        s["q"], s["k"], s["v"] = normal(N, Hk, DIM), normal(N, Hk, DIM), normal(N, H, DIM)
        s["state"] = normal(P, H, DIM, DIM, dtype=DTYPES[case["state"]])
        slots = torch.randperm(P, generator=gen, device=dev)[:N].to(torch.int32)
        slots[N - pad:] = -1
        s["slots"] = slots
        if op == "la_decode":
            s["g"] = decay(N, H) if case["g"] == "token" else decay(H)
        else:
            s["g"] = -5.0 * torch.rand((N, H, DIM), generator=gen, device=dev)
            b = torch.randn((N, H), generator=gen, device=dev)
            s["beta"] = (b if case["logit"] else torch.sigmoid(b)).to(torch.bfloat16)
    elif op == "gated_norm":
        M, H = case["M"], case["H"]
        s["x"], s["gate"] = normal(M, H, DIM), normal(M, H, DIM)
        s["weight"] = 1 + normal(DIM, dtype=DTYPES[case["weight"]], std=0.1)
        if case["act"] == "none":
            s["gate"] = None
    else:
        M, D = case["M"], case["D"]
        s["x"] = normal(M, D)
        s["residual"] = normal(M, D, dtype=DTYPES[case["residual"]])
        s["weight"] = 1 + normal(D, dtype=DTYPES[case["weight"]], std=0.1)
        s["post"] = 1 + normal(D, dtype=DTYPES[case["weight"]], std=0.1) if case["post"] else None
        s["gate"] = normal(D, dtype=DTYPES[case["weight"]], std=0.5) if case["gate"] else None
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import kimi_delta_attention_kda_gb300 as kda
    c = s["case"]
    if c["op"] == "la_prefill":
        return kda.la_prefill(s["q"], s["k"], s["v"], s["g"], init_state=s["init"], cu_seqlens=s.get("cu"),
                              state_dtype=DTYPES[c["state"]])
    if c["op"] == "la_decode":
        return kda.la_decode(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"]), s["state"]
    if c["op"] == "kda_decode":
        out = kda.kda_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"],
                             beta_is_logit=c["logit"])
        return out, s["state"]
    if c["op"] == "gated_norm":
        return kda.gated_norm(s["x"], s["weight"], gate=s["gate"], activation=c["act"], gate_first=c["first"], eps=EPS)
    return kda.residual_norm(s["x"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                             scale=c["scale"], eps=EPS)


# ---------------------------------------------------------------- plain forms

def _run_plain(s):
    op = s["case"]["op"]
    if op == "la_prefill":
        return _plain_la_prefill(s)
    if op == "la_decode":
        return _plain_la_decode(s)
    if op == "kda_decode":
        return _plain_kda_decode(s)
    if op == "gated_norm":
        return _plain_gated_norm(s)
    return _plain_residual_norm(s)


def _plain_la_prefill(s):
    """Chunks of 64 tokens: scores within each chunk, a state for each chunk,
    and the states before the chunks as one product over all chunks."""
    c = s["case"]
    H, dt = c["H"], DTYPES[c["state"]]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    q, k = (x.repeat_interleave(H // x.shape[2], dim=2) for x in (q, k))
    g = s["g"].double().expand(*v.shape[:3])   # sums of decays over long ranges: 64 bits
    if c["packed"]:
        # One row for each sequence, as long as the longest; no decay and no
        # key behind a sequence's end.
        cu = s["cu"]
        N, L = c["B"], max(s["lengths"])
        at = cu[:-1, None] + torch.arange(L, device=cu.device)
        here = at < cu[1:, None]
        at = at.clamp(max=c["T"] - 1)
        q, k, v, g = (torch.where(here.view(N, L, *[1] * (x.dim() - 2)), x[0][at], 0) for x in (q, k, v, g))
    B, T = v.shape[:2]
    n = -(-T // CHUNK)
    pad = n * CHUNK - T

    def chunks(x):   # [B, T, H, d] -> [B, H, n, CHUNK, d]
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], dim=1)
        return x.view(B, n, CHUNK, H, -1).permute(0, 3, 1, 2, 4)

    q, k, v, g = chunks(q), chunks(k), chunks(v), chunks(g.unsqueeze(-1)).squeeze(-1)
    G = g.cumsum(-1)                                                  # within the chunk
    total = G[..., -1]
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    P = (q @ k.mT) * torch.where(causal, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    Z = v.mT @ (k * (total[..., None] - G).exp().float()[..., None])   # [B, H, n, value, key]
    # The state before chunk i: each earlier chunk's Z, decayed over the chunks between.
    S0 = s["init"].float() if s["init"] is not None else torch.zeros(B, H, DIM, DIM, device=q.device)
    Z = torch.cat([S0[:, :, None], Z], dim=2)
    run_total = torch.cat([torch.zeros_like(total[..., :1]), total.cumsum(-1)], dim=-1)
    below = torch.ones(n + 1, n + 1, dtype=torch.bool, device=q.device).tril()
    W = torch.where(below, run_total[..., :, None] - run_total[..., None, :], -math.inf).exp().float()
    S = (W @ Z.flatten(-2)).view(B, H, n + 1, DIM, DIM)
    o = P @ v + (q * G.exp().float()[..., None]) @ S[:, :, :-1].mT
    o = (SCALE * o).permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, DIM)[:, :T]
    if c["packed"]:
        o = o[here][None]
    return o.to(torch.bfloat16), S[:, :, -1].to(dt)


def _plain_slots(s):
    N, pad = s["case"]["N"], s["case"]["pad"]
    return N - pad, s["slots"][:N - pad].long()


def _plain_out(s, rows, o):
    out = torch.zeros_like(s["v"])
    out[:rows] = o.to(torch.bfloat16)
    return out


def _plain_la_decode(s):
    rows, at = _plain_slots(s)
    H = s["case"]["H"]
    q, k, v = (s[x][:rows].float() for x in ("q", "k", "v"))
    q, k = (x.repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
    g = s["g"].expand(s["case"]["N"], H)[:rows]
    S = g.exp()[..., None, None] * s["state"][at].float() + v[..., :, None] * k[..., None, :]
    o = SCALE * (S * q[..., None, :]).sum(-1)
    s["state"][at] = S.to(s["state"].dtype)
    return _plain_out(s, rows, o), s["state"]


def _plain_kda_decode(s):
    rows, at = _plain_slots(s)
    q, k, v, g, b = (s[x][:rows].float() for x in ("q", "k", "v", "g", "beta"))
    if s["case"]["logit"]:
        b = 1 / (1 + (-b).exp())
    q, k = (x * ((x * x).sum(-1, keepdim=True) + 1e-6).rsqrt() for x in (q, k))
    S = s["state"][at].float() * g.exp()[..., None, :]
    u = b[..., None] * (v - (S * k[..., None, :]).sum(-1))
    S = S + u[..., :, None] * k[..., None, :]
    o = SCALE * (S * q[..., None, :]).sum(-1)
    s["state"][at] = S.to(s["state"].dtype)
    return _plain_out(s, rows, o), s["state"]


def _plain_gated_norm(s):
    c = s["case"]
    x, w = s["x"].float(), s["weight"].float()
    a = torch.ones_like(x)
    if s["gate"] is not None:
        z = s["gate"].float()
        a = 1 / (1 + (-z).exp())
        a = a * z if c["act"] == "silu" else a
    if c["first"]:
        x = x * a
    y = x * ((x * x).mean(-1, keepdim=True) + EPS).rsqrt() * w
    if not c["first"]:
        y = y * a
    return y.to(torch.bfloat16)


def _plain_residual_norm(s):
    c = s["case"]
    u = s["x"].float()
    if s["post"] is not None:
        u = u * ((u * u).mean(-1, keepdim=True) + EPS).rsqrt() * s["post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    r = s["residual"].float() + c["scale"] * u
    y = r * ((r * r).mean(-1, keepdim=True) + EPS).rsqrt() * s["weight"].float()
    return y.to(torch.bfloat16), r.to(s["residual"].dtype)


# ---------------------------------------------------------------------- work

def work(case):
    """Bytes: each input once, each output once.  Flops: the recurrence's own
    (4 per state element and token, 6 for KDA's error term), the norms' none
    to speak of."""
    op, H = case["op"], case.get("H")
    state = DIM * DIM * (2 if case.get("state") == "bf16" else 4)
    if op == "la_prefill":
        tokens = case["T"] if case["packed"] else case["B"] * case["T"]
        n = tokens * (512 * (case["Hk"] + H) + (4 * H if case["g"] == "token" else 0))
        n += case["B"] * H * state * (2 if case["init"] else 1)
        return {"bytes": n, "flops": 4 * DIM * DIM * tokens * H}
    if op in ("la_decode", "kda_decode"):
        rows, Hk = case["N"] - case["pad"], case.get("Hk", H)
        n = rows * (2 * H * state + 512 * (Hk + H)) + case["pad"] * H * 256
        n += rows * H * (4 * DIM + 2) if op == "kda_decode" else rows * H * 4
        return {"bytes": n, "flops": (7 if op == "kda_decode" else 5) * DIM * DIM * rows * H}
    if op == "gated_norm":
        rows = case["M"] * H
        return {"bytes": rows * 256 * (2 if case["act"] == "none" else 3), "flops": 12 * rows * DIM}
    n = case["M"] * case["D"]
    return {"bytes": n * (4 + 2 * (2 if case["residual"] == "bf16" else 4)), "flops": 10 * n}


# --------------------------------------------------------- definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {key: x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x for key, x in s.items()}
    op = case["op"]
    if op == "la_prefill":
        return _exact_la_prefill(case, d)
    if op in ("la_decode", "kda_decode"):
        return _exact_step(case, d)
    if op == "gated_norm":
        z = d["gate"]
        a = 1.0 if z is None else torch.sigmoid(z) if case["act"] == "sigmoid" else z * torch.sigmoid(z)
        x = d["x"] * a if case["first"] else d["x"]
        y = d["weight"] * x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        return y if case["first"] else y * a
    rms = lambda x: torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)  # noqa: E731
    x = d["x"] if d["post"] is None else d["post"] * (d["x"] / rms(d["x"]))
    r = d["residual"] + case["scale"] * (x if d["gate"] is None else d["gate"] * x)
    return d["weight"] * (r / rms(r)), r


def _exact_la_prefill(case, d):
    """The recurrence token by token, all sequences at once."""
    H, per = case["H"], case["H"] // case["Hk"]
    cu = [0]
    for n in d["lengths"] if case["packed"] else [case["T"]] * case["B"]:
        cu.append(cu[-1] + n)
    N, longest = len(cu) - 1, max(cu[i + 1] - cu[i] for i in range(len(cu) - 1))
    if longest > 80000 or longest * N * H > (1 << 21):
        return None                              # the plain recurrence would take too long
    flat = lambda x: x.reshape(-1, *x.shape[2:])  # noqa: E731
    q, k, v = flat(d["q"]), flat(d["k"]), flat(d["v"])
    decay = torch.exp(d["g"] if case["g"] == "head" else flat(d["g"]))
    S = d["init"] if d["init"] is not None else v.new_zeros(N, H, DIM, DIM)
    out = torch.empty_like(v)
    start, length = cu[:-1], [cu[i + 1] - cu[i] for i in range(N)]
    order = sorted(range(N), key=lambda i: -length[i])
    S = S[order]                                 # longest first: the live ones are a prefix
    begin = torch.tensor([start[i] for i in order], device=v.device)
    for t in range(longest):
        live = sum(length[i] > t for i in order)
        row = begin[:live] + t
        kt, qt = (x[row].repeat_interleave(per, dim=1) for x in (k, q))
        a = decay.expand(live, H) if case["g"] == "head" else decay[row]
        St = S[:live]
        St.mul_(a[..., None, None]).addcmul_(v[row].unsqueeze(-1), kt.unsqueeze(-2))
        out[row] = torch.einsum("nhvk,nhk->nhv", St, qt) * SCALE
    back = torch.empty_like(S)
    back[order] = S
    return out.view(d["v"].shape), back


def _exact_step(case, d):
    N, H = case["N"] - case["pad"], case["H"]
    at = d["slots"][:N].long()
    pool, out = d["state"], torch.zeros_like(d["v"])
    q, k, v = (d[x][:N] for x in ("q", "k", "v"))
    S = pool[at]
    if case["op"] == "la_decode":
        q, k = (x.repeat_interleave(H // x.shape[1], dim=1) for x in (q, k))
        decay = torch.exp(d["g"] if d["g"].dim() == 1 else d["g"][:N])
        S = S * decay[..., None, None] + torch.einsum("nhv,nhk->nhvk", v, k)
    else:
        unit = lambda x: x / torch.sqrt(x.square().sum(-1, keepdim=True) + 1e-6)  # noqa: E731
        q, k = unit(q), unit(k)
        b = torch.sigmoid(d["beta"][:N]) if case["logit"] else d["beta"][:N]
        S = S * torch.exp(d["g"][:N]).unsqueeze(-2)
        u = (v - torch.einsum("nhvk,nhk->nhv", S, k)) * b.unsqueeze(-1)
        S = S + torch.einsum("nhv,nhk->nhvk", u, k)
    out[:N] = SCALE * torch.einsum("nhvk,nhk->nhv", S, q)
    pool[at] = S
    return out, pool
