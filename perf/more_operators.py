"""Cases for measuring the selective state space scan and the short causal
convolution in front of it, each for whole prompts and for single tokens.

``run`` computes an operator in its plain form (torch, 32 bits) or, with
``own``, through this package; ``exact`` gives the definition in 64 bits.
"""

import math

import torch

own = False

CHUNK = 64                      # tokens per chunk of the plain scan
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HEADS = (1, 2, 3, 5, 6, 8, 12, 16, 32, 48, 64, 96)   # channels: 128 for each


def listed():
    return [
        # The q, k and v of one prompt on a small tensor-parallel shard, going
        # on from an earlier part of it.
        {"name": "conv_prefill t8192 d2304", "op": "conv_prefill", "B": 1, "T": 8192, "D": 2304, "W": 4,
         "packed": False, "act": "silu", "bias": False, "weight": "bf16", "init": True, "fused": False},
        # One half of the input projection of a layer at the full width.
        {"name": "conv_prefill t8192 d12288", "op": "conv_prefill", "B": 1, "T": 8192, "D": 12288, "W": 4,
         "packed": False, "act": "silu", "bias": True, "weight": "fp32", "init": False, "fused": True},
        # A packed batch of ragged prompts: the q, k and v of 12 heads.
        {"name": "conv_prefill packed8 d4608", "op": "conv_prefill", "B": 8, "T": 33333, "D": 4608, "W": 4,
         "packed": True, "act": "silu", "bias": False, "weight": "bf16", "init": True, "fused": False},
        # One conversation on a shard: the latency of a token.
        {"name": "conv_decode n1 d2304", "op": "conv_decode", "N": 1, "D": 2304, "W": 4, "pool": 4, "pad": 0,
         "act": "silu", "bias": False, "weight": "bf16", "fused": False},
        # A serving batch padded to a captured graph's size, q, k and v of 96 heads.
        {"name": "conv_decode n128 d36864", "op": "conv_decode", "N": 128, "D": 36864, "W": 4, "pool": 130, "pad": 3,
         "act": "silu", "bias": True, "weight": "fp32", "fused": True},
        # A prompt of the default benchmark's length on a shard of 768 channels.
        {"name": "ssm_prefill t8192 d768", "op": "ssm_prefill", "B": 1, "T": 8192, "D": 768, "N": 16, "G": 1,
         "packed": False, "dt": "bf16", "bc": "bf16", "gate": True, "skip": True, "state": "fp32", "init": True,
         "fused": True},
        # The same prompt at the full width.
        {"name": "ssm_prefill t8192 d12288", "op": "ssm_prefill", "B": 1, "T": 8192, "D": 12288, "N": 16, "G": 1,
         "packed": False, "dt": "bf16", "bc": "bf16", "gate": True, "skip": True, "state": "fp32", "init": False,
         "fused": True},
        # A packed batch of ragged prompts.
        {"name": "ssm_prefill packed8 d1536", "op": "ssm_prefill", "B": 8, "T": 33333, "D": 1536, "N": 16, "G": 1,
         "packed": True, "dt": "bf16", "bc": "bf16", "gate": True, "skip": True, "state": "bf16", "init": True,
         "fused": True},
        # Larger states, two groups of channels with keys of their own, step sizes kept in FP32.
        {"name": "ssm_prefill b2 t2000 d1536 n64", "op": "ssm_prefill", "B": 2, "T": 2000, "D": 1536, "N": 64, "G": 2,
         "packed": False, "dt": "fp32", "bc": "fp32", "gate": False, "skip": True, "state": "fp32", "init": True,
         "fused": False},
        # Short prompts: latency.
        {"name": "ssm_prefill b3 t77 d768", "op": "ssm_prefill", "B": 3, "T": 77, "D": 768, "N": 16, "G": 1,
         "packed": False, "dt": "bf16", "bc": "bf16", "gate": True, "skip": True, "state": "fp32", "init": False,
         "fused": True},
        {"name": "ssm_decode n1 d768", "op": "ssm_decode", "N": 1, "D": 768, "S": 16, "G": 1, "pool": 4, "pad": 0,
         "dt": "bf16", "bc": "bf16", "gate": True, "skip": True, "state": "fp32", "fused": True},
        {"name": "ssm_decode n128 d12288", "op": "ssm_decode", "N": 128, "D": 12288, "S": 16, "G": 1, "pool": 130,
         "pad": 3, "dt": "bf16", "bc": "bf16", "gate": True, "skip": True, "state": "fp32", "fused": True},
    ]


def _log(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n - 1 if n % 1024 == 0 else n


def draw(rng):
    op = rng.choice(("conv_prefill", "conv_decode", "ssm_prefill", "ssm_prefill", "ssm_decode"))
    D = 128 * rng.choice(HEADS) if rng.random() < 0.7 else _log(rng, 1, 12288)
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("conv"):
        D *= rng.choice((1, 3))
        case = {"op": op, "D": D, "W": rng.choice((2, 3, 4, 4, 4)), "act": rng.choice(("silu", "silu", "none")),
                "bias": flip(), "weight": rng.choice(("fp32", "bf16")), "fused": flip()}
        if op == "conv_decode":
            N = _log(rng, 1, min(1024, 128 * 36864 // D))
            return {**case, "N": N, "pool": N + rng.randint(0, 5), "pad": min(N - 1, rng.randint(0, 3))}
        T = _log(rng, 1, min(65536, 8192 * 12288 // D))
        B = _log(rng, 1, max(1, min(32, 8192 * 12288 // (D * T))))
        packed = flip()
        return {**case, "B": B, "T": B * T if packed else T, "packed": packed, "init": flip()}
    S = rng.choice((5, 8, 16, 16, 16, 32, 64))
    G = rng.choice([x for x in (1, 1, 1, 2, 4) if D % x == 0])
    kinds = {"dt": rng.choice(("bf16", "bf16", "fp32")), "bc": rng.choice(("bf16", "bf16", "fp32")),
             "gate": rng.random() < 0.7, "skip": flip(), "state": rng.choice(("fp32", "bf16")), "fused": flip()}
    if op == "ssm_decode":
        N = _log(rng, 1, max(1, min(1024, 128 * 12288 * 16 // (D * max(S, 16)))))
        return {"op": op, "N": N, "D": D, "S": S, "G": G, "pool": N + rng.randint(0, 5),
                "pad": min(N - 1, rng.randint(0, 3)), **kinds}
    most = 8192 * 12288 * 16 // (D * max(S, 16))
    T = _log(rng, 1, min(65536, most))
    B = _log(rng, 1, max(1, min(32, most // T)))
    packed = flip()
    return {"op": op, "B": B, "T": B * T if packed else T, "D": D, "N": S, "G": G, "packed": packed, "init": flip(),
            **kinds}


def _lengths(case, seed):
    """Each sequence's tokens: ragged whole numbers that add up to T in a packed batch."""
    B, T = case["B"], case["T"]
    if not case["packed"]:
        return [T] * B
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, T + 1, (B - 1,), generator=gen).sort().values.tolist()
    ends = [0] + cuts + [T]
    return [ends[i + 1] - ends[i] for i in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (std * torch.randn(shape, generator=gen, device=dev)).to(dtype)

    def part(lead, width, before, after, dtype=torch.bfloat16):
        """Channels of a wider projection's output where the case is fused."""
        if not case["fused"]:
            before = after = 0
        return normal(*lead, before + width + after, dtype=dtype)[..., before:before + width]

    s = {"case": dict(case)}
    op, D = case["op"], case["D"]
    decode = op.endswith("decode")
    if decode:
        N, pool, pad = case["N"], case["pool"], case["pad"]
        lead = (N,)
        slots = torch.randperm(pool, generator=gen, device=dev)[:N].to(torch.int32)
        slots[N - pad:] = -1
        s["slots"] = slots
    else:
        N = case["B"]
        lead = (1, case["T"]) if case["packed"] else (N, case["T"])
        s["lengths"] = _lengths(case, seed)
        if case["packed"]:
            s["cu"] = torch.tensor([0] + s["lengths"], device=dev).cumsum(0)
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = part(lead, D, 0, D)
        s["weight"] = normal(D, W, dtype=DTYPES[case["weight"]], std=W ** -0.5)
        s["bias"] = normal(D, dtype=DTYPES[case["weight"]], std=0.1) if case["bias"] else None
        if decode:
            s["state"] = normal(pool, W - 1, D)
        else:
            s["init"] = normal(N, W - 1, D) if case["init"] else None
        return s
    S, G = case["S"] if decode else case["N"], case["G"]
    s["x"] = torch.nn.functional.silu(normal(*lead, D))
    rank = -(-D // 16)
    s["dt"] = normal(*lead, D, dtype=DTYPES[case["dt"]])
    # Step sizes softplus(dt + bias) from about 1/1000 to about 1, as layers are initialised.
    step = torch.exp(math.log(1e-3) + math.log(100) * torch.rand(D, generator=gen, device=dev))
    s["dt_bias"] = torch.log(torch.expm1(step))
    # Rates 1 .. S, spread by a fifth.
    s["A"] = -torch.arange(1, S + 1, device=dev) * torch.exp(normal(D, S, dtype=torch.float32, std=0.2))
    bc = part(lead, 2 * G * S, rank, 0, dtype=DTYPES[case["bc"]])
    s["B"], s["C"] = (y.unflatten(-1, (G, S)) for y in bc.split(G * S, dim=-1))
    if not case["fused"]:
        s["B"], s["C"] = s["B"].contiguous(), s["C"].contiguous()
    s["z"] = part(lead, D, D, 0) if case["gate"] else None
    s["D"] = 1 + normal(D, dtype=torch.float32, std=0.1) if case["skip"] else None
    if decode:
        s["state"] = normal(pool, D, S, dtype=DTYPES[case["state"]])
    else:
        s["init"] = normal(N, D, S, dtype=DTYPES[case["state"]]) if case["init"] else None
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import kimi_delta_attention_kda_gb300 as kda
    c = s["case"]
    if c["op"] == "conv_prefill":
        return kda.conv_prefill(s["x"], s["weight"], bias=s["bias"], init_state=s["init"], cu_seqlens=s.get("cu"),
                                activation=c["act"])
    if c["op"] == "conv_decode":
        out = kda.conv_decode(s["x"], s["weight"], s["state"], bias=s["bias"], slots=s["slots"], activation=c["act"])
        return out, s["state"]
    if c["op"] == "ssm_prefill":
        return kda.ssm_prefill(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                               init_state=s["init"], cu_seqlens=s.get("cu"), state_dtype=DTYPES[c["state"]])
    out = kda.ssm_decode(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"],
                         dt_bias=s["dt_bias"], slots=s["slots"])
    return out, s["state"]


# ---------------------------------------------------------------- plain forms

def _run_plain(s):
    op = s["case"]["op"]
    if op == "conv_prefill":
        return _plain_conv_prefill(s)
    if op == "conv_decode":
        return _plain_conv_decode(s)
    if op == "ssm_prefill":
        return _plain_ssm_prefill(s)
    return _plain_ssm_decode(s)


def _silu(x):
    return x / (1 + (-x).exp())


def _taps(s, rows):
    """rows [..., W, D], oldest first, through the filter."""
    y = (rows.float() * s["weight"].float().t()).sum(-2)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return (_silu(y) if s["case"]["act"] == "silu" else y).to(torch.bfloat16)


def _plain_conv_prefill(s):
    """Every token's W rows by index, from the initial states and the tokens in one table."""
    c, x = s["case"], s["x"]
    N, W, D = c["B"], c["W"], c["D"]
    flat = x.reshape(-1, D)
    init = s["init"] if s["init"] is not None else torch.zeros(N, W - 1, D, dtype=x.dtype, device=x.device)
    table = torch.cat([init.reshape(-1, D), flat])
    length = s["cu"].diff() if c["packed"] else torch.full((N,), c["T"], device=x.device)
    start = length.cumsum(0) - length
    seq = torch.arange(N, device=x.device).repeat_interleave(length, output_size=flat.shape[0])

    def row(n, at):
        """Where the table has position `at` of sequence n (below 0: its initial state)."""
        return torch.where(at < 0, n * (W - 1) + at + W - 1, N * (W - 1) + start[n] + at)

    back = torch.arange(1 - W, 1, device=x.device)
    at = torch.arange(flat.shape[0], device=x.device) - start[seq]
    out = _taps(s, table[row(seq[:, None], at[:, None] + back)])
    n = torch.arange(N, device=x.device)[:, None]
    final = table[row(n, length[:, None] + back[:-1])]
    return out.view(x.shape), final


def _plain_conv_decode(s):
    rows, at = s["case"]["N"] - s["case"]["pad"], s["slots"].long()
    window = torch.cat([s["state"][at[:rows]], s["x"][:rows, None]], dim=1)
    out = torch.zeros(s["x"].shape, dtype=torch.bfloat16, device=s["x"].device)
    out[:rows] = _taps(s, window)
    s["state"][at[:rows]] = window[:, 1:]
    return out, s["state"]


def _steps(s):
    """softplus(dt + bias) in FP32: max(u, 0) + log(1 + exp(-|u|))."""
    u = s["dt"].float() + s["dt_bias"]
    return u.clamp(min=0) + (-u.abs()).exp().log1p()


def _finish(s, y, x):
    """The skip of x and the gate, rounded once."""
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(torch.bfloat16)


def _plain_ssm_prefill(s):
    """Chunks of 64 tokens, one position of every chunk at a time: first from
    zero states, then, with the states before the chunks known, for the outputs."""
    c = s["case"]
    A, D, S = s["A"], c["D"], c["N"]
    x, dt = s["x"].float(), _steps(s)
    groups = lambda y: y.float().repeat_interleave(D // c["G"], dim=2)  # noqa: E731
    Bm, Cm = (y.float() if c["G"] == 1 else groups(y) for y in (s["B"], s["C"]))   # [B, T, 1 or D, S]
    full = s["x"]
    if c["packed"]:
        # One row for each sequence, as long as the longest; no step behind a sequence's end.
        cu = s["cu"]
        N, L = c["B"], max(s["lengths"])
        at = cu[:-1, None] + torch.arange(L, device=cu.device)
        here = at < cu[1:, None]
        at = at.clamp(max=c["T"] - 1)
        x, dt, Bm, Cm = (torch.where(here.view(N, L, *[1] * (y.dim() - 2)), y[0][at], 0) for y in (x, dt, Bm, Cm))
    N, T = x.shape[:2]
    n = -(-T // CHUNK)

    def chunks(y):   # [N, T, ...] -> [CHUNK, N * n, ...]
        y = torch.cat([y, y.new_zeros(N, n * CHUNK - T, *y.shape[2:])], dim=1)
        return y.view(N * n, CHUNK, *y.shape[2:]).transpose(0, 1).contiguous()

    x_in = x
    u, dt, Bm, Cm = chunks(dt * x), chunks(dt), chunks(Bm), chunks(Cm)

    def walk(h, y):
        for t in range(CHUNK):
            h = (dt[t][..., None] * A).exp_().mul_(h).add_(u[t][..., None] * Bm[t])
            if y is not None:
                torch.sum(h * Cm[t], dim=-1, out=y[t])
        return h

    h = walk(x.new_zeros(N * n, D, S), None).view(N, n, D, S)
    total = dt.sum(0).view(N, n, D)
    S0 = s["init"].float() if s["init"] is not None else torch.zeros(N, D, S, device=x.device)
    before = []
    for i in range(n):
        before.append(S0)
        S0 = (total[:, i, :, None] * A).exp() * S0 + h[:, i]
    y = torch.empty(CHUNK, N * n, D, device=x.device)
    walk(torch.stack(before, dim=1).view(N * n, D, S), y)
    y = y.transpose(0, 1).reshape(N, n * CHUNK, D)[:, :T]
    if c["packed"]:
        y, x_in = y[here][None], full.float()
    return _finish(s, y, x_in), S0.to(DTYPES[c["state"]])


def _plain_ssm_decode(s):
    c = s["case"]
    rows = c["N"] - c["pad"]
    at = s["slots"][:rows].long()
    x, dt = s["x"].float(), _steps(s)
    Bm, Cm = (y[:rows].float().repeat_interleave(c["D"] // c["G"], dim=1) for y in (s["B"], s["C"]))
    h = (dt[:rows, :, None] * s["A"]).exp() * s["state"][at].float() + (dt * x)[:rows, :, None] * Bm
    y = torch.zeros_like(x)
    y[:rows] = (h * Cm).sum(-1)
    out = _finish(s, y, x)
    out[rows:] = 0
    s["state"][at] = h.to(s["state"].dtype)
    return out, s["state"]


# ---------------------------------------------------------------------- work

def work(case):
    """Bytes: each input once, each output once.  Flops: 2 for each tap of the
    filter; for each token, channel and state 7 (the decay's product and
    exponential, the update's two products and sum, the output's two)."""
    op, D = case["op"], case["D"]
    size = lambda kind: 4 if case[kind] == "fp32" else 2  # noqa: E731
    if op == "conv_prefill":
        W, tokens = case["W"], case["T"] if case["packed"] else case["B"] * case["T"]
        n = 4 * tokens * D + D * (W + case["bias"]) * size("weight")
        n += case["B"] * (W - 1) * D * 2 * (2 if case["init"] else 1)
        return {"bytes": n, "flops": 2 * W * tokens * D}
    if op == "conv_decode":
        W, rows = case["W"], case["N"] - case["pad"]
        n = rows * D * (4 + 4 * (W - 1)) + case["pad"] * D * 2 + D * (W + case["bias"]) * size("weight")
        return {"bytes": n, "flops": 2 * W * rows * D}
    S, G = case["S"] if op == "ssm_decode" else case["N"], case["G"]
    if op == "ssm_decode":
        rows = case["N"] - case["pad"]
        n, states = case["pad"] * D * 2, 2 * rows
    else:
        rows = case["T"] if case["packed"] else case["B"] * case["T"]
        n, states = 0, case["B"] * (2 if case["init"] else 1)
    n += rows * (D * (4 + size("dt") + (2 if case["gate"] else 0)) + 2 * G * S * size("bc"))
    n += states * D * S * size("state") + 4 * D * (S + 1 + case["skip"])
    return {"bytes": n, "flops": 7 * S * D * rows}


# --------------------------------------------------------- definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    d = {key: x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x for key, x in s.items()}
    op = case["op"]
    if op == "conv_prefill":
        return _exact_conv_prefill(case, d)
    if op == "conv_decode":
        return _exact_conv_decode(case, d)
    if op == "ssm_prefill":
        return _exact_ssm_prefill(case, d)
    return _exact_ssm_decode(case, d)


def _exact_conv_prefill(case, d):
    """Sequence by sequence, the filter as a sum of shifted products."""
    W, D = case["W"], case["D"]
    x = d["x"].reshape(-1, D)
    out, finals, at = torch.empty_like(x), [], 0
    for n, length in enumerate(d["lengths"]):
        head = d["init"][n] if d["init"] is not None else x.new_zeros(W - 1, D)
        rows = torch.cat([head, x[at:at + length]])
        y = torch.zeros_like(rows[:length])
        for j in range(W):
            y += rows[j:j + length] * d["weight"][:, j]
        if d["bias"] is not None:
            y += d["bias"]
        out[at:at + length] = y * torch.sigmoid(y) if case["act"] == "silu" else y
        finals.append(rows[length:])
        at += length
    return out.view(d["x"].shape), torch.stack(finals)


def _exact_conv_decode(case, d):
    out, pool = torch.zeros_like(d["x"]), d["state"]
    at = d["slots"][:case["N"] - case["pad"]].long()
    y = d["x"][:len(at)] * d["weight"][:, -1] + torch.einsum("nwd,dw->nd", pool[at], d["weight"][:, :-1])
    if d["bias"] is not None:
        y = y + d["bias"]
    out[:len(at)] = torch.nn.functional.silu(y) if case["act"] == "silu" else y
    pool[at] = torch.cat([pool[at][:, 1:], d["x"][:len(at), None]], dim=1)
    return out, pool


def _exact_dt(d):
    u = d["dt"] + d["dt_bias"]
    return torch.logaddexp(u, torch.zeros_like(u))


def _exact_ssm_prefill(case, d):
    """The recurrence token by token, all sequences at once."""
    D, S, G = case["D"], case["N"], case["G"]
    length = d["lengths"]
    N, longest = len(length), max(length)
    if longest > 80000:
        return None                              # the plain recurrence would take too long
    flat = lambda y: y.reshape(-1, *y.shape[2:])  # noqa: E731
    x, dt, Bm, Cm = flat(d["x"]), flat(_exact_dt(d)), flat(d["B"]), flat(d["C"])
    order = sorted(range(N), key=lambda i: -length[i])
    start = [sum(length[:i]) for i in order]
    begin = torch.tensor(start, device=x.device)
    h = d["init"][order] if d["init"] is not None else x.new_zeros(N, D, S)
    h = h.view(N, G, D // G, S)
    A = d["A"].view(G, D // G, S)
    y = torch.empty_like(x)
    for t in range(longest):
        live = sum(n > t for n in length)        # longest first: the live ones are a prefix
        row = begin[:live] + t
        step = dt[row].view(live, G, -1, 1)
        now = h[:live]
        now.mul_(torch.exp(step * A)).addcmul_(step * x[row].view(live, G, -1, 1), Bm[row].unsqueeze(2))
        y[row] = (now @ Cm[row].unsqueeze(-1)).view(live, D)
    if d["D"] is not None:
        y += x * d["D"]
    if d["z"] is not None:
        y *= torch.nn.functional.silu(flat(d["z"]))
    back = torch.empty(N, D, S, dtype=h.dtype, device=h.device)
    back[order] = h.view(N, D, S)
    return y.view(d["x"].shape), back


def _exact_ssm_decode(case, d):
    D, S, G = case["D"], case["S"], case["G"]
    at = d["slots"][:case["N"] - case["pad"]].long()
    n = len(at)
    x, dt = d["x"][:n], _exact_dt(d)[:n]
    split = lambda y: y.view(*y.shape[:-1], G, D // G)  # noqa: E731
    h = d["state"][at].view(n, G, D // G, S)
    h = h * torch.exp(torch.einsum("ngd,gds->ngds", split(dt), d["A"].view(G, D // G, S)))
    h = h + torch.einsum("ngd,ngs->ngds", split(dt * x), d["B"][:n])
    y = torch.einsum("ngds,ngs->ngd", h, d["C"][:n]).reshape(n, D)
    if d["D"] is not None:
        y = y + d["D"] * x
    if d["z"] is not None:
        y = y * d["z"][:n] * torch.sigmoid(d["z"][:n])
    out = torch.zeros_like(d["x"])
    out[:n] = y
    d["state"][at] = h.view(n, D, S)
    return out, d["state"]
