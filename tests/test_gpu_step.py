"""kda_la_decode and kda_decode against one token of their recurrences in 64 bits.

Bounds: every product and sum is FP32, with sums of 128 terms and a few
roundings beside them: 2^-16 of a value's magnitude; out adds one BF16
rounding, and so does a BF16 state.
"""

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

D = 128
TYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


def draw(N, H, Hk, pool, delta, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = {"q": rnd(N, Hk, D).bfloat16(), "k": rnd(N, Hk, D).bfloat16(), "v": rnd(N, H, D).bfloat16(),
         "g": -5 * torch.rand((N, H, D) if delta else (N, H), generator=gen),
         "state": rnd(pool, H, D, D).to(dtype)}
    if delta:
        d["beta"] = rnd(N, H).bfloat16()
    return d, gen


def check(kda, d, slots, delta, logit=False, status=0):
    N, pool = d["v"].shape[0], d["state"].shape[0]
    at = list(range(N)) if slots is None else slots
    dev = {key: x.cuda() for key, x in d.items()}
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    if delta:
        out = kda.kda_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], dev["state"], slots=sl,
                             beta_is_logit=logit)
    else:
        out = kda.la_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["state"], slots=sl)
    torch.cuda.synchronize()
    assert kda.device_status() == status
    rows = [i for i in range(N) if 0 <= at[i] < pool]
    S = d["state"][[at[i] for i in rows]]
    pick = {key: x if key == "g" and x.dim() == 1 else x[rows] for key, x in d.items() if key != "state"}
    if delta:
        beta = pick["beta"]
        o, s, oa, sa = ref.kda_step(pick["q"], pick["k"], pick["v"], pick["g"], beta, S, logit)
    else:
        o, s, oa, sa = ref.la_step(pick["q"], pick["k"], pick["v"], pick["g"], S)
    new, out = dev["state"].cpu(), out.cpu()
    ref.assert_close(out[rows], o, ref.HALF_BF16 * o.abs() + 2.0 ** -16 * oa, "out")
    half = ref.HALF_BF16 if new.dtype == torch.bfloat16 else 0.0
    ref.assert_close(new[[at[i] for i in rows]], s, half * s.abs() + 2.0 ** -16 * sa, "state")
    rest = [p for p in range(pool) if p not in {at[i] for i in rows}]
    assert torch.equal(new[rest], d["state"][rest])
    off = [i for i in range(N) if i not in rows]
    assert not out[off].any()


@pytest.mark.parametrize("N,H,Hk", [(1, 1, 1), (1, 6, 6), (3, 12, 4), (7, 5, 5), (30, 6, 2), (40, 8, 8)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("per_head", [False, True])
def test_la_step(kda, N, H, Hk, dtype, per_head):
    d, gen = draw(N, H, Hk, N + 3, False, N * H, dtype)
    if per_head:
        d["g"] = d["g"][0].contiguous()
    check(kda, d, torch.randperm(N + 3, generator=gen)[:N].tolist(), False)


@pytest.mark.parametrize("N,H", [(1, 1), (1, 6), (3, 12), (7, 5), (30, 6), (40, 8)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("logit", [False, True])
def test_kda_step(kda, N, H, dtype, logit):
    d, gen = draw(N, H, H, N + 3, True, N * H, dtype)
    if not logit:
        d["beta"] = torch.sigmoid(d["beta"].float()).bfloat16()
    check(kda, d, torch.randperm(N + 3, generator=gen)[:N].tolist(), True, logit)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("N", [4, 60])
def test_padding_rows_and_no_slots(kda, delta, N):
    d, _ = draw(N, 3, 3, N + 1, delta, 3, torch.float32)
    check(kda, d, None, delta, True)
    d, _ = draw(N, 3, 3, N + 1, delta, 4, torch.bfloat16)
    check(kda, d, [-1, 2, -7] + [N - i for i in range(N - 3)], delta, True)
    d["state"] = d["state"][:0]
    check(kda, d, [-1] * N, delta, True)


@pytest.mark.parametrize("delta", [False, True])
def test_slot_beyond_the_pool(kda, delta):
    """The host cannot see it: the kernel's own check makes it padding."""
    d, _ = draw(3, 2, 2, 4, delta, 5, torch.float32)
    check(kda, d, [0, 4, 3], delta, True, status=8)
    check(kda, d, [2 ** 31 - 1, 1, -2 ** 31], delta, True, status=8)


def test_no_sequences(kda):
    e = torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    st = torch.ones(2, 2, D, D, device="cuda")
    assert kda.la_decode(e, e, e, torch.empty(0, 2, device="cuda"), st).shape == (0, 2, D)
    assert kda.kda_decode(e, e, e, torch.empty(0, 2, D, device="cuda"), torch.empty_like(e[..., 0]), st).numel() == 0
    assert (st == 1).all()


@pytest.mark.parametrize("delta", [False, True])
def test_extreme_decays_and_zero_vectors(kda, delta):
    d, _ = draw(5, 2, 2, 5, delta, 6, torch.float32)
    d["g"][0] = float("-inf")
    d["g"][1] = 0.0
    d["g"][2] = -200.0
    d["k"][3] = 0
    d["q"][4] = 0
    check(kda, d, None, delta, True)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite_rows_stay_apart(kda, delta, dtype):
    d, _ = draw(4, 2, 2, 4, delta, 7, dtype)
    d["v"][1, 1, 9] = float("nan")
    d["k"][2, 0, 3] = float("inf")
    d["state"][3, 1, 4, 4] = float("nan")
    check(kda, d, [1, 0, 3, 2], delta, True)


def test_prefill_then_steps(kda):
    """A prompt, then single tokens, against the longer prompt: both operators."""
    gen = torch.Generator().manual_seed(8)
    T, more, H = 133, 5, 4
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v = (rnd(1, T + more, H, D).bfloat16().cuda() for _ in range(3))
    gl = (-0.3 * torch.rand((1, T + more, H), generator=gen)).cuda()
    o, f, oa, fa = ref.la_tokens(q.cpu(), k.cpu(), v.cpu(), gl.cpu())
    _, st = kda.la_prefill(q[:, :T].contiguous(), k[:, :T].contiguous(), v[:, :T].contiguous(),
                           gl[:, :T].contiguous())
    for t in range(T, T + more):
        out = kda.la_decode(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(),
                            gl[:, t].contiguous(), st)
        ref.assert_close(out[0], o[0, t], ref.HALF_BF16 * o[0, t].abs() + 2.0 ** -13 * oa[0, t], "la token %d" % t)
    ref.assert_close(st, f, 2.0 ** -13 * fa, "la state")
    # kda: the whole prompt in one call, and the split one.
    g = (-5 * torch.rand((1, T + more, H, D), generator=gen)).cuda()
    b = torch.sigmoid(rnd(1, T + more, H)).bfloat16().cuda()
    whole, _ = kda.kda_prefill(q, k, v, g, b)
    cut = lambda x: x[:, :T].contiguous()  # noqa: E731
    _, st = kda.kda_prefill(cut(q), cut(k), cut(v), cut(g), cut(b))
    st = st.float()
    for t in range(T, T + more):
        one = lambda x: x[:, t].contiguous()  # noqa: E731
        out = kda.kda_decode(one(q), one(k), one(v), one(g), one(b), st)
        # kda_prefill's own tolerance (rel. 1e-2), on both sides.
        assert (out[0].float() - whole[0, t].float()).norm() <= 2e-2 * whole[0, t].float().norm()


@pytest.mark.parametrize("delta", [False, True])
def test_graph(kda, delta):
    """A captured step advances the states at every replay."""
    d, _ = draw(5, 3, 3, 6, delta, 9, torch.float32)
    dev = {key: x.cuda() for key, x in d.items()}
    slots = torch.tensor([4, 0, -1, 5, 2], dtype=torch.int32, device="cuda")
    out = torch.empty_like(dev["v"])

    def call(state):
        if delta:
            return kda.kda_decode(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], state, slots=slots, out=out,
                                  beta_is_logit=True)
        return kda.la_decode(dev["q"], dev["k"], dev["v"], dev["g"], state, slots=slots, out=out)

    want = dev["state"].clone()
    for _ in range(3):
        call(want)
    last = out.clone()
    state = dev["state"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(state)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, want) and torch.equal(out, last)
