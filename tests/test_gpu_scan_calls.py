"""The convolution's and the scan's calls on CUDA tensors: what they turn away,
what came just before them in the streams, several at once, and the run of them
together that a layer makes."""

import threading

import pytest
import torch

import ops_reference as ref
import scan_reference as scan

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


def bf(*s):
    return torch.zeros(s, dtype=BF16, device="cuda")


def f32(*s):
    return torch.zeros(s, device="cuda")


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device="cuda")


GOOD = {
    "conv_prefill": lambda: dict(x=bf(2, 9, 24), weight=bf(24, 4), bias=bf(24), init_state=bf(2, 3, 24), out=bf(2, 9, 24),
                                 final_state=bf(2, 3, 24)),
    "conv_decode": lambda: dict(x=bf(3, 24), weight=f32(24, 3), state=bf(5, 2, 24), bias=f32(24),
                                slots=torch.arange(3, dtype=torch.int32, device="cuda"), out=bf(3, 24)),
    "ssm_prefill": lambda: dict(x=bf(2, 9, 24), dt=bf(2, 9, 24), A=f32(24, 16), B=bf(2, 9, 2, 16), C=bf(2, 9, 2, 16),
                                D=f32(24), z=bf(2, 9, 24), dt_bias=f32(24), init_state=f32(2, 24, 16), out=bf(2, 9, 24),
                                final_state=f32(2, 24, 16)),
    "ssm_decode": lambda: dict(x=bf(3, 24), dt=f32(3, 24), A=f32(24, 16), B=f32(3, 2, 16), C=f32(3, 2, 16), D=f32(24),
                               z=bf(3, 24), dt_bias=f32(24), state=bf(5, 24, 16),
                               slots=torch.arange(3, dtype=torch.int32, device="cuda"), out=bf(3, 24)),
}
OPTIONAL = {"bias", "init_state", "out", "final_state", "slots", "D", "z", "dt_bias"}


@pytest.mark.parametrize("op,name", [(op, name) for op in GOOD for name in {
    "conv_prefill": "x weight bias init_state out final_state", "conv_decode": "x weight state bias slots out",
    "ssm_prefill": "x dt A B C D z dt_bias init_state out final_state",
    "ssm_decode": "x dt A B C D z dt_bias state slots out"}[op].split()])
def test_each_argument(kda, op, name):
    call = getattr(kda, op)
    call(**GOOD[op]())
    good = GOOD[op]()[name]
    strided = torch.zeros(good.shape[:-1] + (2 * good.shape[-1],), dtype=good.dtype, device="cuda")[..., ::2]
    bad = [good.double(), good.half(), good.cpu(), strided, good.new_zeros(good.shape + (1,)), good[..., :-1].contiguous()]
    if name != "state":
        bad.append(good.new_zeros((good.shape[0] + 1,) + good.shape[1:]))
    if name in ("x", "dt", "B", "C", "z"):   # rows that do not lie at one distance, or overlap
        bad += [good.new_zeros(good.shape[-1:]).expand(good.shape)]
        if good.dim() >= 3 and op.endswith("prefill"):
            bad += [good.new_zeros((good.shape[0], good.shape[1] + 1) + good.shape[2:])[:, 1:],
                    good.transpose(0, 1).contiguous().transpose(0, 1)]
    before = {key: t.clone() for key, t in GOOD[op]().items()}
    for t in bad:
        args = GOOD[op]()
        args[name] = t
        with pytest.raises(ValueError):
            call(**args)
        for key, value in args.items():
            if key != name:
                assert torch.equal(value, before[key])
    args = GOOD[op]()
    args[name] = None
    if name in OPTIONAL:
        call(**args)
    else:
        with pytest.raises((ValueError, AttributeError)):
            call(**args)
    torch.cuda.synchronize()
    assert kda.device_status() == 0


def test_values(kda):
    a = GOOD["conv_prefill"]()
    with pytest.raises(ValueError, match="activation"):
        kda.conv_prefill(**a, activation="sigmoid")
    with pytest.raises(ValueError, match="2 to 4"):
        kda.conv_prefill(a["x"], bf(24, 5))
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.conv_prefill(bf(1, 9, 24), a["weight"], cu_seqlens=i32(2))
    with pytest.raises(ValueError, match="B == 1"):
        kda.conv_prefill(a["x"], a["weight"], cu_seqlens=torch.tensor([0, 18], device="cuda"))
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(bf(1, 0, 24), a["weight"], cu_seqlens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    b = GOOD["conv_decode"]()
    with pytest.raises(ValueError, match="fewer rows"):
        kda.conv_decode(bf(9, 24), b["weight"], b["state"])
    c = GOOD["ssm_prefill"]()
    with pytest.raises(ValueError, match="states"):
        kda.ssm_prefill(c["x"], c["dt"], c["A"], c["B"], c["C"], state_dtype=torch.float16)
    with pytest.raises(ValueError, match="C must"):
        kda.ssm_prefill(c["x"], c["dt"], c["A"], c["B"], c["C"].float())
    with pytest.raises(ValueError, match="groups"):
        kda.ssm_prefill(c["x"], c["dt"], c["A"], bf(2, 9, 5, 16), bf(2, 9, 5, 16))
    with pytest.raises(ValueError, match="1 to 64"):
        kda.ssm_prefill(c["x"], c["dt"], f32(24, 65), bf(2, 9, 2, 65), bf(2, 9, 2, 65))
    d = GOOD["ssm_decode"]()
    d["slots"], d["state"] = None, bf(2, 24, 16)
    with pytest.raises(ValueError, match="fewer rows"):
        kda.ssm_decode(**d)
    # Overlapping outputs are the library's to refuse.
    for op, name in (("conv_prefill", "x"), ("conv_decode", "x"), ("ssm_prefill", "z"), ("ssm_decode", "x")):
        args = GOOD[op]()
        args["out"] = args[name]
        with pytest.raises(kda.KdaError):
            getattr(kda, op)(**args)
    # A wide row's unused part is nobody else's to write.
    wide = bf(2, 9, 48)
    with pytest.raises(kda.KdaError):
        kda.conv_prefill(wide[..., :24], a["weight"], out=wide.view(-1)[:432].view(2, 9, 24))


def test_truth_values(kda):
    class Odd:
        def __bool__(self):
            raise RuntimeError("no truth value")
    c = GOOD["ssm_prefill"]()
    for kw in (dict(dt_softplus=Odd()), dict(output_final_state=Odd())):
        c["out"].fill_(3)
        with pytest.raises(RuntimeError, match="no truth value"):
            kda.ssm_prefill(**c, **kw)
        assert (c["out"] == 3).all()


def inputs(T, dim, N, seed, packed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    lead = (1, N * T) if packed else (N, T)
    return {"x": rnd(*lead, dim).bfloat16(), "dt": rnd(*lead, dim).bfloat16(), "B": rnd(*lead, 1, 16).bfloat16(),
            "C": rnd(*lead, 1, 16).bfloat16(), "z": rnd(*lead, dim).bfloat16(), "A": -torch.exp(rnd(dim, 16)),
            "D": rnd(dim), "dt_bias": rnd(dim) - 3, "init_state": rnd(N, dim, 16), "weight": rnd(dim, 4),
            "conv_init": rnd(N, 3, dim).bfloat16()}


def layer(kda, at, cu):
    """The convolution's output is the scan's x."""
    x, conv_state = kda.conv_prefill(at["x"], at["weight"], init_state=at["conv_init"], cu_seqlens=cu)
    y, state = kda.ssm_prefill(x, at["dt"], at["A"], at["B"], at["C"], at["D"], at["z"], at["dt_bias"],
                               init_state=at["init_state"], cu_seqlens=cu)
    return x, conv_state, y, state


@pytest.mark.parametrize("last", ["x", "dt", "B", "z", "init_state", "conv_init"])
@pytest.mark.parametrize("T,N,packed", [(2100, 1, False), (100, 2, False), (1050, 2, True), (1, 1200, True)])
def test_inputs_rewritten_just_before(kda, T, N, packed, last):
    """Two sets of inputs in turn in the same buffers, `last` written last.  Equal
    bits to calls with a pause before and after each, eagerly and in a graph."""
    dim = 96
    sets = [inputs(T, dim, N, seed, packed) for seed in range(2)]
    at = {key: torch.empty_like(x) for key, x in sets[0].items()}
    cu = torch.arange(0, N * T + 1, T, device="cuda") if packed else None
    order = [key for key in at if key != last] + [last]

    def chain(pause):
        results = []
        for i in range(4):
            for key in order:
                at[key].copy_(sets[i % 2][key])
            if pause:
                torch.cuda.synchronize()
            results.append(layer(kda, at, cu))
            if pause:
                torch.cuda.synchronize()
        return results

    want = chain(True)
    assert not torch.equal(want[0][2], want[1][2])

    def same(got):
        return all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))

    for _ in range(3):
        assert same(chain(False))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(2):
        for outputs in got:
            for x in outputs:
                x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got)
    assert kda.device_status() == 0


def test_inputs_from_another_stream(kda):
    """A call behind a wait for an event of another stream, whose late copies are its inputs."""
    src = inputs(2100, 96, 1, 3, False)
    at = {key: torch.zeros_like(x) for key, x in src.items()}
    big = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    want = layer(kda, src, None)
    torch.cuda.synchronize()
    for _ in range(3):
        for x in at.values():
            x.zero_()
        layer(kda, at, None)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = big
            for _ in range(12):
                y = y @ big
            for key in at:
                at[key].copy_(src[key])
        torch.cuda.current_stream().wait_stream(side)
        got = layer(kda, at, None)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        side.wait_stream(torch.cuda.current_stream())


def test_calls_from_several_threads(kda):
    """Calls at once on streams of their own, and a pool of states that each thread has for itself."""
    def work(seed):
        at, results = inputs(600, 160, 2, seed, False), []
        conv_pool, pool = at["conv_init"].clone(), at["init_state"].clone()
        for t in range(15):
            results += layer(kda, at, None)
            x = kda.conv_decode(at["x"][:, t], at["weight"], conv_pool)
            results.append(kda.ssm_decode(x, at["dt"][:, t], at["A"], at["B"][:, t], at["C"][:, t], pool, at["D"],
                                          at["z"][:, t], at["dt_bias"]))
        torch.cuda.current_stream().synchronize()
        return results + [conv_pool, pool]

    alone = [work(seed) for seed in range(4)]
    got = [None] * 4

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = work(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    for want, have in zip(alone, got):
        assert have is not None and all(torch.equal(x, y) for x, y in zip(want, have))


def test_layer_against_its_definition(kda):
    """The run together, as a layer makes it: parts of one projection through the
    convolution and the scan over a packed batch, and then tokens one by one on
    the pools of states, against both definitions."""
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dim, S, lengths, more = 64, 16, (70, 3, 45), 4
    N, T = len(lengths), sum(lengths)
    cu = [0, 70, 73, 118]
    wide, keys, dt = rnd(1, T, 2 * dim).bfloat16(), rnd(1, T, 5 + 2 * S).bfloat16(), rnd(1, T, dim).bfloat16()
    w, bias, A, D, step = rnd(dim, 4) / 2, rnd(dim) / 4, -torch.exp(rnd(dim, S)), rnd(dim), rnd(dim) - 3
    g = lambda t: t.cuda()  # noqa: E731
    wide_g, keys_g, cu_g = g(wide), g(keys), torch.tensor(cu, device="cuda")
    part = lambda t, i: t[..., 5 + S * i:5 + S * (i + 1)].unflatten(-1, (1, S))  # noqa: E731
    x, conv_state = kda.conv_prefill(wide_g[..., :dim], g(w), g(bias), cu_seqlens=cu_g)
    y, state = kda.ssm_prefill(x, g(dt), g(A), part(keys_g, 0), part(keys_g, 1), g(D), wide_g[..., dim:], g(step),
                               cu_seqlens=cu_g)
    want_x, want_conv, off_x = scan.conv(wide[..., :dim], w, bias, None, cu)
    ref.assert_close(x, want_x, off_x + scan.rounded(want_x, BF16), "x")
    assert torch.equal(conv_state.cpu(), want_conv.bfloat16())
    # From the x that the library has: its rounding is the convolution's.
    o, f, oe, fe = scan.scan(x.cpu(), dt, A, part(keys, 0), part(keys, 1), D, wide[..., dim:], step, cu=cu)
    ref.assert_close(y, o, oe + scan.rounded(o, BF16), "y")
    ref.assert_close(state, f, fe, "state")
    slots = [4, 0, 2]
    conv_pool, pool = bf(6, 3, dim), f32(6, dim, S)
    conv_pool[slots], pool[slots] = conv_state, state
    slots_g = torch.tensor(slots + [-1], dtype=torch.int32, device="cuda")
    for _ in range(more):
        wide, keys, dt = rnd(N + 1, 2 * dim).bfloat16(), rnd(N + 1, 5 + 2 * S).bfloat16(), rnd(N + 1, dim).bfloat16()
        wide_g, keys_g = g(wide), g(keys)
        before_conv, before = conv_pool[slots].cpu(), pool[slots].cpu()
        x = kda.conv_decode(wide_g[..., :dim], g(w), conv_pool, g(bias), slots_g)
        y = kda.ssm_decode(x, g(dt), g(A), part(keys_g, 0), part(keys_g, 1), pool, g(D), wide_g[..., dim:], g(step),
                           slots=slots_g)
        want_x, want_conv, off_x = scan.conv(wide[:N, None, :dim], w, bias, before_conv)
        ref.assert_close(x[:N, None], want_x, off_x + scan.rounded(want_x, BF16), "x")
        assert torch.equal(conv_pool[slots].cpu(), want_conv.bfloat16())
        o, f, oe, fe = scan.scan(x[:N, None].cpu(), dt[:N, None], A, part(keys, 0)[:N, None], part(keys, 1)[:N, None], D,
                                 wide[:N, None, dim:], step, init=before, cut=0.0)
        ref.assert_close(y[:N, None], o, oe + scan.rounded(o, BF16), "y")
        ref.assert_close(pool[slots], f, fe, "state")
        assert not x[N].any() and not y[N].any()
    assert not pool[[1, 3, 5]].any() and not conv_pool[[1, 3, 5]].any()


def test_launches(kda):
    from kimi_delta_attention_kda_gb300 import _lib
    for T, N, packed, want in ((100, 1, False, 1), (2100, 1, False, 2), (1, 1200, True, 3), (1, 1024, True, 2)):
        at = inputs(T, 96, N, 1, packed)
        cu = torch.arange(0, N * T + 1, T, device="cuda") if packed else None
        kda.conv_prefill(at["x"], at["weight"], cu_seqlens=cu)
        assert _lib.last_call_launches() == (2 if N > 1024 else 1)
        kda.ssm_prefill(at["x"], at["dt"], at["A"], at["B"], at["C"], cu_seqlens=cu)
        assert _lib.last_call_launches() == want, (T, N)
