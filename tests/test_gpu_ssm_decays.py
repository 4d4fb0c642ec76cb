"""The decays of kda_ssm_prefill and kda_ssm_decode at their edges: steps that differ from token
to token, rates without bound, growing states, and states that last for thousands of tokens."""

import pytest
import torch

import ops_reference as ref
import scan_reference as scan
from test_gpu_ssm import BF16, F32, check, cuts, draw, kda, on_gpu, want_of  # noqa: F401

pytestmark = pytest.mark.gpu


def decayed(kda, dt, A, init):  # noqa: F811
    """What is left of the initial states [1, dim, S] behind steps dt [1, T, dim] alone."""
    zero = torch.zeros(dt.shape, dtype=BF16, device="cuda")
    keys = torch.zeros(1, dt.shape[1], 1, A.shape[1], dtype=BF16, device="cuda")
    return kda.ssm_prefill(zero, dt.cuda(), A.cuda(), keys, keys, init_state=init.cuda(), dt_softplus=False)[1]


def left(dt, A, init):
    return init.double() * torch.exp(dt.double().sum(1)[..., None] * A.double())


@pytest.mark.parametrize("phase", [0, 5, 15, 16, 31])
@pytest.mark.parametrize("T,step,other", [(8192, 2.5e-3, 0.0), (8192, 2.6e-3, 1e-9), (16384, 1e-4, 0.0)])
def test_one_step_in_32(kda, T, step, other, phase):  # noqa: F811
    """Steps that count at one token of every 32 (the others' decays are 1 in FP32).  Each rounds its decay
    and its product by at most 2^-24, uncorrelated, and the exponential is off by at
    most 3e-8 on average: nothing that is made up for may add more than that."""
    gen = torch.Generator().manual_seed(phase)
    dim, S = 96, 16
    dt = torch.full((1, T, dim), other)
    dt[:, phase::32] = step * (0.9 + 0.2 * torch.rand(1, T // 32, dim, generator=gen))
    A, init = -(0.9 + 0.2 * torch.rand(dim, S, generator=gen)), 1 + torch.rand(1, dim, S, generator=gen)
    n = T // 32
    for on in (False, True):
        kda.set_segments(on, 0)
        off = decayed(kda, dt, A, init).cpu().double() / left(dt, A, init) - 1
        assert off.pow(2).mean().sqrt() < 2.0 ** -24 * (n * 2 / 3) ** 0.5 + 3e-8 * n


def test_small_arguments(kda):  # noqa: F811
    """The mean over many states: their roundings (1.6e-6 each, as test_slow_states has them) cancel to
    5 x 1.6e-6 / sqrt(96 x 16) < 2.1e-7, and the exponential's mean error, 5e-9 to 1e-8 here, is
    made up for to 4e-9."""
    gen = torch.Generator().manual_seed(2)
    T, dim, S = 1024, 96, 16
    dt = 1e-3 * (0.5 + torch.rand(1, T, dim, generator=gen))
    A, init = -(0.7 + 0.6 * torch.rand(dim, S, generator=gen)), 1 + torch.rand(1, dim, S, generator=gen)
    for on in (False, True):
        kda.set_segments(on, 0)
        off = decayed(kda, dt, A, init).cpu().double() / left(dt, A, init) - 1
        assert off.mean().abs() < 2.1e-7 + 4e-9 * T


@pytest.mark.parametrize("S", [16, 32, 64])
def test_infinite_states_stay(kda, S):  # noqa: F811
    """Where no step is taken an infinite state stays one, and with a step that decays it too."""
    for T, step in ((200, 0.0), (200, 1e-3)):
        init = torch.ones(1, 40, S)
        init[0, 3, 1], init[0, 7, 0] = float("inf"), float("-inf")
        for on, chunks in ((False, 0), (True, 4)):
            kda.set_segments(on, chunks)
            fin = decayed(kda, torch.full((1, T, 40), step), -torch.ones(40, S), init).cpu()
            assert torch.equal(torch.isinf(fin), torch.isinf(init)) and torch.equal(fin.sign(), init.sign())


@pytest.mark.parametrize("rate", [float("-inf"), torch.finfo(F32).min])
@pytest.mark.parametrize("S", [16, 5, 8, 32, 64])
@pytest.mark.parametrize("state", [F32, BF16])
@pytest.mark.parametrize("softplus", [False, True])
def test_single_tokens_without_a_step(kda, rate, S, state, softplus):  # noqa: F811
    """A step of zero leaves the states as they are, whatever the rates; any other step leaves
    nothing of states whose rate has no bound."""
    N, dim = 6, 40
    d = on_gpu(draw((N,), dim, S, S, dt=F32, init=N, state=state, bias=False))
    pool = d.pop("init_state")
    d["A"][3] = d["A"][17, 0] = rate
    d["dt"][:] = -200.0 if softplus else 0.0   # softplus(-200) is 0 in FP32
    before = pool.clone()
    out = kda.ssm_decode(**d, state=pool, dt_softplus=softplus)
    assert torch.equal(pool, before) and torch.isfinite(out).all()
    d["dt"].fill_(0.5)
    d["A"][3] = d["A"][17, 0] = -1e30
    want_pool = pool.clone()
    want = kda.ssm_decode(**d, state=want_pool, dt_softplus=softplus)
    d["A"][3] = d["A"][17, 0] = rate
    got = kda.ssm_decode(**d, state=pool, dt_softplus=softplus)
    assert torch.equal(got, want) and torch.equal(pool, want_pool) and torch.isfinite(pool).all()


@pytest.mark.parametrize("S", [16, 5, 64])
def test_growing_states(kda, S):  # noqa: F811
    """Rates above zero, and steps below it, over spans in which an exponential of the whole
    growth would not be finite: states of zero stay zero, and what has grown is a number
    where the tokens one by one give one."""
    T, dim = 2048, 40
    d = draw((1, T), dim, S, 5, dt=F32, init=1, bias=False, z=False)
    gen = torch.Generator().manual_seed(3)
    d["dt"] = 0.2 * (0.9 + 0.2 * torch.rand(1, T, dim, generator=gen))
    # Even channels: a rate above 0, nothing but zeros up to the last 100 tokens.
    d["A"][0::2] = 1.0
    d["x"][:, :-100, 0::2] = 0
    d["init_state"][:, 0::2] = 0
    # Odd ones: 512 tokens grow from 1e-30 by about exp(102), as many take it back, and so on;
    # of four channels by exp(-102) first.
    d["A"][1::2] = -1.0
    sign = torch.ones(T)
    sign[:512] = sign[1024:1536] = -1
    d["dt"][:, :, 1::2] *= sign[:, None]
    d["x"][:, :, 1::2] = 0
    d["dt"][:, :, 1:9:2] *= -1
    d["init_state"][:, 1:9:2] *= 1e30
    d["init_state"][:, 9::2] *= 1e-30
    want = want_of(d, softplus=False)
    assert torch.isfinite(want[1]).all()
    for on, chunks in ((False, 0), (True, 32), (True, 0)):
        kda.set_segments(on, chunks)
        check(kda, d, softplus=False, want=want)


def test_long_conversations(kda):  # noqa: F811
    """2000 single tokens on FP32 states that only decay: bounds as in test_small_arguments and
    test_slow_states."""
    gen = torch.Generator().manual_seed(4)
    T, N, dim, S = 2000, 2, 64, 16
    for mean in (1e-3, 1e-2):
        dt = mean * (0.5 + torch.rand(T, N, dim, generator=gen))
        A, init = -(0.7 + 0.6 * torch.rand(dim, S, generator=gen)), 1 + torch.rand(N, dim, S, generator=gen)
        pool, dev, A_dev = init.cuda(), dt.cuda(), A.cuda()
        zero, keys = torch.zeros(N, dim, dtype=BF16, device="cuda"), torch.zeros(N, 1, S, dtype=BF16, device="cuda")
        for t in range(T):
            kda.ssm_decode(zero, dev[t], A_dev, keys, keys, pool, dt_softplus=False)
        want = init.double() * torch.exp(dt.double().sum(0)[..., None] * A.double())
        off = pool.cpu().double() / want - 1
        rms = 2.0 ** -24 * (T * 2 / 3) ** 0.5
        assert off.mean().abs() < 5 * rms / (N * dim * S) ** 0.5 + (4e-9 if mean < 2e-3 else 1e-8) * T
        assert off.pow(2).mean().sqrt() < rms + 1e-8 * T


def test_infinite_states_stay_in_pools(kda):  # noqa: F811
    """As test_infinite_states_stay, for single tokens."""
    for step in (0.0, 1e-3):
        pool = torch.ones(3, 40, 16, device="cuda")
        pool[0, 3, 1], pool[2, 7, 0] = float("inf"), float("-inf")
        before = pool.clone()
        zero, keys = torch.zeros(3, 40, dtype=BF16, device="cuda"), torch.zeros(3, 1, 16, dtype=BF16, device="cuda")
        for _ in range(3):
            kda.ssm_decode(zero, zero.float() + step, -torch.ones(40, 16, device="cuda"), keys, keys, pool, dt_softplus=False)
        assert torch.equal(torch.isinf(pool), torch.isinf(before)) and torch.equal(pool.sign(), before.sign())


@pytest.mark.parametrize("S", [1, 3, 5, 8, 16, 20, 24, 48, 64])
@pytest.mark.parametrize("bc", [BF16, F32])
def test_infinite_inputs(kda, S, bc):  # noqa: F811
    """An infinite x or step gives infinite states and outputs where the definition does, not NaN,
    whatever the length of a row of states."""
    T, dim = 150, 40
    d = draw((1, T), dim, S, S, dt=F32, bc=bc, init=1, z=False, D=False)
    d["B"], d["C"] = d["B"].abs() + 1, d["C"].abs() + 1
    d["A"] = -torch.arange(1, S + 1).expand(dim, S).contiguous() / 64.0
    d["x"][0, 10, 3], d["x"][0, 60, 5] = float("inf"), float("-inf")
    d["dt"][0, 12, 7], d["x"][0, 12, 7] = float("inf"), 1.0

    def same(got, want, what):
        for kind in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(kind(got).cpu(), kind(want)), what
    o, f, _, _ = want_of(d)
    assert torch.isposinf(o[0, 12:, [3, 7]]).all() and torch.isneginf(o[0, 60:, 5]).all()
    for on, chunks in ((False, 0), (True, 4)):
        kda.set_segments(on, chunks)
        out, fin = kda.ssm_prefill(**on_gpu(d))
        same(out, o, "out")
        same(fin, f, "final")
    for state in (F32, BF16):
        dev = on_gpu(d)
        pool = dev.pop("init_state").to(state)
        for t in range(70):
            one = {key: v[:, t] if key in ("x", "dt", "B", "C") and v is not None else v for key, v in dev.items()}
            same(kda.ssm_decode(**one, state=pool), o[:, t], "token %d" % t)
