"""kda_ssm_prefill and kda_ssm_decode against the recurrence in 64 bits; bounds
as scan_reference.py derives them."""

import pytest
import torch

import ops_reference as ref
import scan_reference as scan

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


@pytest.fixture(autouse=True)
def cuts(kda):
    yield
    kda.set_segments(True, 0)


def draw(lead, dim, S, seed, G=1, dt=BF16, bc=BF16, z=True, D=True, bias=True, init=None, state=F32, part=0):
    """part: every row is a part of a wider one, `part` elements from its start."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731

    def row(width, dtype):
        return rnd(*lead, part + width + (part and 3)).to(dtype)[..., part:part + width]
    d = {"x": row(dim, BF16), "dt": row(dim, dt), "B": row(G * S, bc).unflatten(-1, (G, S)),
         "C": row(G * S, bc).unflatten(-1, (G, S)), "z": row(dim, BF16) if z else None,
         "A": -torch.exp(rnd(dim, S)) * torch.arange(1, S + 1) / 4, "D": rnd(dim) if D else None,
         "dt_bias": rnd(dim) - 3 if bias else None,
         "init_state": rnd(init, dim, S).to(state) if init else None}
    return d


def on_gpu(d):
    """The tensors there, parts of wider rows as they are here."""
    def put(t):
        if t is None:
            return None
        wide = torch.empty_strided((t.untyped_storage().nbytes() // t.element_size(),), (1,), dtype=t.dtype)
        wide.set_(t.untyped_storage(), 0, wide.shape, (1,))
        return wide.cuda().as_strided(t.shape, t.stride(), t.storage_offset())
    return {key: put(t) for key, t in d.items()}


def want_of(d, cu=None, softplus=True, **kw):
    return scan.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["z"], d["dt_bias"], softplus,
                     d["init_state"], cu, **kw)


def check(kda, d, cu=None, softplus=True, want=None, **kw):
    dev = on_gpu(d)
    cu_dev = None if cu is None else torch.tensor(cu, device="cuda")
    out, fin = kda.ssm_prefill(**dev, cu_seqlens=cu_dev, dt_softplus=softplus, **kw)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    o, f, oe, fe = want_of(d, cu, softplus) if want is None else want
    ref.assert_close(out, o, oe + scan.rounded(o, BF16), "out")
    ref.assert_close(fin, f, fe + scan.rounded(f, fin.dtype), "final")
    return out, fin


@pytest.mark.parametrize("B,T,dim", [(1, 1, 1), (1, 2, 8), (2, 3, 33), (1, 31, 32), (1, 32, 40), (3, 77, 96), (1, 300, 257)])
@pytest.mark.parametrize("S", [1, 5, 16, 17, 32, 64])
def test_fixed(kda, B, T, dim, S):
    check(kda, draw((B, T), dim, S, T * dim + S))
    check(kda, draw((B, T), dim, S, T * dim + S + 1, dt=F32, bc=F32, z=False, D=False, init=B))
    check(kda, draw((B, T), dim, S, T * dim + S + 2, bias=False, init=B, state=BF16))


@pytest.mark.parametrize("dim,G", [(64, 2), (96, 3), (72, 2), (30, 5), (40, 40)])
@pytest.mark.parametrize("S", [16, 6])
def test_groups(kda, dim, G, S):
    check(kda, draw((2, 70), dim, S, dim, G=G, init=2))


@pytest.mark.parametrize("part", [1, 2, 3, 4, 8, 16])
@pytest.mark.parametrize("S", [16, 8, 3])
def test_part_of_wider_rows(kda, part, S):
    check(kda, draw((2, 45), 40, S, part, part=part, G=2))
    check(kda, draw((2, 45), 32, S, part, part=part, dt=F32, bc=F32))


def test_no_softplus(kda):
    d = draw((1, 90), 40, 16, 1, bias=False)
    d["dt"] = d["dt"].abs()
    check(kda, d, softplus=False)
    d = draw((1, 90), 40, 16, 2, dt=F32)
    d["dt"] = d["dt"].abs() + 3.5
    # A channel whose steps are negative grows by up to exp(90 |step|) a token: beyond FP32's range
    # (2^128 = exp(88.7)) within a few tokens, where the 64 bits still have a number.
    out, fin = kda.ssm_prefill(**on_gpu(d), dt_softplus=False, state_dtype=BF16)
    o, f, oe, fe = want_of(d, softplus=False)
    grows = (d["dt"] + d["dt_bias"] < 0).any(1)[0]
    assert 0 < grows.sum() < 20
    ref.assert_close(out.cpu()[..., ~grows], o[..., ~grows], (oe + scan.rounded(o, BF16))[..., ~grows], "out")
    ref.assert_close(fin.cpu()[:, ~grows], f[:, ~grows], (fe + scan.rounded(f, BF16))[:, ~grows], "final")


LENGTHS = [[5], [0, 7], [1] * 9, [3, 0, 0, 40, 2, 129, 0], [64, 64, 64], [31, 33, 1, 95], [0, 0, 3], [300, 1, 0, 200]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("dim,S", [(40, 16), (33, 7), (32, 64)])
def test_packed(kda, lengths, dim, S):
    """Whole, and in spans of 32, 64 and 96 tokens."""
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    for init, state in ((None, F32), (len(lengths), F32), (len(lengths), BF16)):
        d = draw((1, cu[-1]), dim, S, cu[-1] + dim, init=init, state=state)
        want = want_of(d, cu)
        for on, chunks in ((True, 0), (False, 0), (True, 1), (True, 4), (True, 5)):
            kda.set_segments(on, chunks)
            check(kda, d, cu, want=want)


@pytest.mark.parametrize("B,T", [(1, 64), (1, 65), (2, 300), (3, 129)])
@pytest.mark.parametrize("dim,S", [(40, 16), (33, 7), (32, 32)])
def test_spans(kda, B, T, dim, S):
    for init in (None, B):
        d = draw((B, T), dim, S, T + dim, init=init)
        want = want_of(d)
        for on, chunks in ((True, 0), (False, 0), (True, 1), (True, 2), (True, 4), (True, 1 << 20)):
            kda.set_segments(on, chunks)
            check(kda, d, want=want)


def test_plan(kda):
    assert kda.ssm_plan_segments(1, 100, 768, 1, 16, False) == 0
    assert kda.ssm_workspace_bytes(1, 100, 768, 1, 16, False) == 0
    n = kda.ssm_plan_segments(1, 8192, 768, 1, 16, False)
    assert n > 4
    need = kda.ssm_workspace_bytes(1, 8192, 768, 1, 16, False)
    assert n * 768 * 17 * 4 <= need <= (n + 1) * 768 * 17 * 4 + 1024
    kda.set_segments(False)
    assert kda.ssm_plan_segments(1, 8192, 768, 1, 16, False) == 0
    kda.set_segments(True, 4)
    assert kda.ssm_plan_segments(2, 8192, 768, 1, 16, False) == 128
    assert kda.ssm_plan_segments(2, 100, 768, 1, 16, True) == 2


def test_long(kda):
    """Slow decays over a long prompt: against the recurrence in 64 bits on the GPU."""
    T, dim, S = 8192, 96, 16
    d = draw((1, T), dim, S, 3)
    d["A"] = d["A"] / 64
    dev = on_gpu(d)
    A, s = dev["A"].double(), scan.steps(dev["dt"], dev["dt_bias"], True)[0]
    x, B, C = dev["x"][0].double(), dev["B"][0].double(), dev["C"][0].double()
    h, E = (torch.zeros(dim, S, dtype=torch.float64, device="cuda") for _ in range(2))
    y = torch.empty(T, dim, dtype=torch.float64, device="cuda")
    for t in range(T):
        a, add = torch.exp(s[t][:, None] * A), (s[t] * x[t])[:, None] * B[t]
        E = a * E + a * h.abs() + add.abs()
        h = a * h + add
        y[t] = (h * C[t]).sum(-1)
    y = (y + dev["D"].double() * x) * scan.silu(dev["z"][0].double())
    for on in (True, False):
        kda.set_segments(on)
        out, fin = kda.ssm_prefill(**dev)
        # E as in scan_reference.py; |dt + dt_bias| stays below 8 here, so a step costs at most
        # 8 (2^-24 + 2^-23) + 2^-21.5 < 2^-19.  out: BF16 roundings of up to 2^-8, 1.7e-3 of the norm over
        # a binade, and h cut to TF32, 2^-11 on average and always towards 0.
        assert (fin[0].double() - h).norm() <= 2.0 ** -19 * E.norm()
        assert (out[0].double() - y).norm() <= (1.7e-3 + 2.0 ** -11 + 2.0 ** -12) * y.norm()


def test_no_tokens(kda):
    for lead, cu, n in (((2, 0), None, 2), ((1, 0), [0, 0, 0, 0], 3)):
        d = draw(lead, 40, 16, 4, init=n, state=BF16)
        out, fin = kda.ssm_prefill(**on_gpu(d), cu_seqlens=None if cu is None else torch.tensor(cu, device="cuda"))
        assert out.numel() == 0 and torch.equal(fin.cpu(), d["init_state"])
        d["init_state"] = None
        out, fin = kda.ssm_prefill(**on_gpu(d), cu_seqlens=None if cu is None else torch.tensor(cu, device="cuda"))
        assert fin.shape == (n, 40, 16) and fin.dtype == F32 and not fin.any()
    out, fin = kda.ssm_prefill(**on_gpu(draw((1, 5), 8, 16, 4)), output_final_state=False)
    assert fin is None and out.shape == (1, 5, 8)


@pytest.mark.parametrize("cu", [[0, 50, 40, 90], [1, 50, 90], [0, 50, 80], [0, 120, 90], [-1, 4, 90]])
@pytest.mark.parametrize("chunks", [0, 1])
def test_bad_offsets(kda, cu, chunks):
    """The host cannot see them: nothing is written."""
    kda.set_segments(True, chunks)
    dev = on_gpu(draw((1, 90), 40, 16, 5))
    out = torch.full((1, 90, 40), 3.0, dtype=BF16, device="cuda")
    fin = torch.full((len(cu) - 1, 40, 16), 3.0, device="cuda")
    kda.ssm_prefill(**dev, cu_seqlens=torch.tensor(cu, device="cuda"), out=out, final_state=fin)
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert (out == 3).all() and (fin == 3).all()


@pytest.mark.parametrize("chunks", [0, 4])
@pytest.mark.parametrize("bad", [False, True])
def test_many_sequences(kda, bad, chunks):
    """More offsets than a CTA checks by itself."""
    kda.set_segments(True, chunks)
    gen = torch.Generator().manual_seed(6)
    cu = [0] + torch.randint(0, 4, (1500,), generator=gen).cumsum(0).tolist()
    d = draw((1, cu[-1]), 8, 4, 7, init=1500)
    if not bad:
        check(kda, d, cu)
        return
    cu[700] = cu[701] + 1
    out = torch.full(d["x"].shape, 3.0, dtype=BF16, device="cuda")
    kda.ssm_prefill(**on_gpu(d), cu_seqlens=torch.tensor(cu, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert kda.device_status() == 1 and (out == 3).all()


@pytest.mark.parametrize("on,chunks", [(True, 0), (False, 0), (True, 2)])
def test_states_in_place(kda, on, chunks):
    kda.set_segments(on, chunks)
    for lead, cu in (((2, 500), None), ((1, 500), [0, 2, 260, 260, 500])):
        n = lead[0] if cu is None else len(cu) - 1
        dev = on_gpu(draw(lead, 40, 16, 8, init=n))
        cu_dev = None if cu is None else torch.tensor(cu, device="cuda")
        want = kda.ssm_prefill(**dev, cu_seqlens=cu_dev)
        again = kda.ssm_prefill(**dev, cu_seqlens=cu_dev)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
        got = kda.ssm_prefill(**dev, cu_seqlens=cu_dev, final_state=dev["init_state"])
        assert got[1] is dev["init_state"] and all(torch.equal(a, b) for a, b in zip(got, want))


def test_far_rows(kda):
    """Rows whose offsets pass 32 bits."""
    d = draw((1, 70), 16, 16, 9)
    dev = on_gpu(d)
    want = kda.ssm_prefill(**dev)
    wide = torch.empty(1, 70, 1 << 25, dtype=BF16, device="cuda")
    at = 0
    for key in ("x", "dt", "B", "C", "z"):
        flat = dev[key].flatten(2)
        view = wide[..., at:at + flat.shape[-1]]
        view.copy_(flat)
        dev[key] = view.unflatten(-1, dev[key].shape[2:])
        at += 64
    got = kda.ssm_prefill(**dev)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("chunks", [0, 2])
@pytest.mark.parametrize("packed", [False, True])
def test_not_finite_stays_apart(kda, value, chunks, packed):
    """What is not finite in a token's x reaches its channel's later tokens alone; in
    its B, its group's; in its C, that token's outputs of the group."""
    kda.set_segments(True, chunks)
    d = draw((2, 100), 64, 16, 10, G=2)
    if packed:
        for key in ("x", "dt", "B", "C", "z"):
            d[key] = d[key].reshape(1, 200, *d[key].shape[2:])
    clean = kda.ssm_prefill(**on_gpu(d), cu_seqlens=torch.tensor([0, 100, 200], device="cuda") if packed else None)
    d["x"].view(-1, 64)[30, 3] = value
    d["C"].view(-1, 2, 16)[20, 0, 2] = value
    d["B"].view(-1, 2, 16)[170, 1, 1] = value
    out, fin = kda.ssm_prefill(**on_gpu(d), cu_seqlens=torch.tensor([0, 100, 200], device="cuda") if packed else None)
    o, clean_o = out.view(200, 64), clean[0].view(200, 64)
    touched = torch.zeros(200, 64, dtype=torch.bool)
    touched[30:100, 3] = True
    touched[20, :32] = True
    touched[170:, 32:] = True
    assert torch.equal(torch.isfinite(o.float()).cpu(), ~touched)
    assert torch.equal(o.cpu()[~touched], clean_o.cpu()[~touched])
    states = torch.isfinite(fin).cpu()
    assert not states[0, 3].any() and not states[1, 32:, 1].any()
    states[0, 3] = states[1, 32:, 1] = True
    assert states.all()


def test_large_and_small_steps(kda):
    """Steps that forget the state, and softplus far from 0."""
    d = draw((1, 64), 40, 16, 11, dt=F32, init=1)
    d["dt_bias"] = None
    d["dt"][0, :, 0] = 16.0
    d["dt"][0, :, 1] = -16.0
    d["dt"][0, :, 2] = 0.0
    d["A"][3] = 0.0
    d["A"][4] = -1e30
    check(kda, d)
    d["dt"][0, :, 5] = 1e4
    d["dt"][0, :, 6] = -1e4
    o, f = kda.ssm_prefill(**on_gpu(d))
    want = want_of(d)
    assert torch.isfinite(o.float()).all()
    assert torch.allclose(f[0, 5:7].cpu().double(), want[1][0, 5:7], rtol=1e-5, atol=0)


@pytest.mark.parametrize("dim,G", [(36, 1), (44, 1), (72, 2), (132, 3)])
@pytest.mark.parametrize("S", [4, 12, 16, 20, 48])
@pytest.mark.parametrize("dt,bc", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_last_channels(kda, dim, G, S, dt, bc):
    """Groups that are no whole 32 channels: whole, in spans, packed, and in place."""
    d = draw((1, 140), dim, S, dim + S, G=G, dt=dt, bc=bc, init=1)
    want = want_of(d)
    for on, chunks in ((False, 0), (True, 4)):
        kda.set_segments(on, chunks)
        out, fin = check(kda, d, want=want)
        dev = on_gpu(d)
        got = kda.ssm_prefill(**dev, final_state=dev["init_state"])
        assert torch.equal(got[0], out) and torch.equal(dev["init_state"], fin)
    cu = [0, 3, 64, 64, 140]
    check(kda, draw((1, 140), dim, S, dim + S, G=G, dt=dt, bc=bc, z=False, init=4, state=BF16), cu)


@pytest.mark.parametrize("dim,S,B,T,cu", [
    (5000, 16, 1, 2100, None), (2500, 16, 3, 700, None), (10300, 64, 1, 530, None), (6000, 5, 1, 1111, None),
    (9000, 32, 1, 1300, [0, 128, 128, 400, 401, 1290, 1300, 1300]), (12200, 16, 1, 3333, [0, 1, 3000, 3333])])
@pytest.mark.parametrize("state", [F32, BF16])
def test_wide(kda, dim, S, B, T, cu, state):
    """More chains than SMs: the bits of the same channels a few at a time, and in
    place, captured and replayed likewise."""
    kda.set_segments(False, 0)
    n = B if cu is None else len(cu) - 1
    d = on_gpu(draw((B, T), dim, S, dim, init=n, state=state))
    if cu is not None:
        d["cu_seqlens"] = torch.tensor(cu, device="cuda")
    out, fin = kda.ssm_prefill(**d)
    for lo in range(0, dim, 1000):
        hi = min(dim, lo + 1000)
        part = {key: t if key in ("B", "C", "cu_seqlens") else t[lo:hi] if key in ("A", "D", "dt_bias") else
                t[:, lo:hi].contiguous() if key == "init_state" else t[..., lo:hi] for key, t in d.items()}
        got = kda.ssm_prefill(**part)
        assert torch.equal(got[0], out[..., lo:hi]) and torch.equal(got[1], fin[:, lo:hi])
    kda.set_segments(True, 0)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        kept = d["init_state"].clone()
        graph = torch.cuda.CUDAGraph()
        d["out"] = torch.empty_like(out)
        with torch.cuda.graph(graph, stream=stream):
            kda.ssm_prefill(**d, final_state=d["init_state"])
        want = kda.ssm_prefill(**{**d, "out": None})
        for _ in range(3):
            d["init_state"].copy_(kept)
            d["out"].zero_()
            graph.replay()
            stream.synchronize()
            assert torch.equal(d["out"], want[0]) and torch.equal(d["init_state"], want[1])
    assert kda.device_status() == 0


@pytest.mark.parametrize("T,dim", [(4000, 128), (1645, 128), (600, 768), (1100, 5000), (2100, 10300)])
@pytest.mark.parametrize("packed", [False, True])
def test_scratch_as_it_was_left(kda, T, dim, packed):
    """What calls before left in the scratch is not read: their numbers are 1e30."""
    d = on_gpu(draw((1, T), dim, 16, T))
    if packed:
        d["cu_seqlens"] = torch.tensor([0, T], device="cuda")
    kda.set_segments(False, 0)
    want = kda.ssm_prefill(**d)
    kda.set_segments(True, 0)
    for before in (512, 12200):
        big = on_gpu(draw((1, 4096), 512, 16, 1))
        big["x"] *= 1e30
        if before > 512:
            big = {k: t.repeat(24, 1) if k == "A" else t.repeat(24) if k in ("D", "dt_bias") else
                   t.repeat(1, 1, 24) if k in ("x", "dt", "z") else t for k, t in big.items()}
        kda.ssm_prefill(**big)
        out, fin = kda.ssm_prefill(**d)
        # A span's state comes by fewer and other products than the walk's; both are off by 2^-18 or so.
        assert torch.allclose(fin, want[1], rtol=1e-4, atol=1e-5)
        assert torch.allclose(out.float(), want[0].float(), rtol=2 ** -6, atol=2e-3)


def test_wide_ones_at_once(kda):
    """Calls whose spans wait for one another, on three streams at the same time: two
    of them as captured graphs, and a call cut into spans beside them."""
    calls = [on_gpu(draw((1, 1500), dim, 16, dim, init=1)) for dim in (5000, 10300, 600)]
    want = [kda.ssm_prefill(**d) for d in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [(torch.empty_like(o), torch.empty_like(f)) for o, f in want]
    graphs = []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            kda.ssm_prefill(**calls[i], out=outs[i][0], final_state=outs[i][1])
    for _ in range(5):
        for o, f in outs:
            o.zero_(), f.zero_()
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            kda.ssm_prefill(**calls[2], out=outs[2][0], final_state=outs[2][1])
        torch.cuda.synchronize()
        assert kda.device_status() == 0
        for got, right in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(got, right))


@pytest.mark.parametrize("rate", [float("-inf"), torch.finfo(F32).min])
@pytest.mark.parametrize("S", [16, 5, 32])
def test_rates_without_bound(kda, rate, S):
    """States that no step keeps, as with a rate of -1e30, also behind the last token."""
    for chunks, cu in ((0, None), (1, None), (0, [0, 37, 37, 45, 77]), (1, [0, 37, 37, 45, 77])):
        kda.set_segments(True, chunks)
        d = on_gpu(draw((1, 77), 40, S, S, init=4 if cu else 1))
        cu = None if cu is None else torch.tensor(cu, device="cuda")
        d["A"][3] = d["A"][17, 1] = -1e30
        want = kda.ssm_prefill(**d, cu_seqlens=cu)
        d["A"][3] = d["A"][17, 1] = rate
        assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(kda.ssm_prefill(**d, cu_seqlens=cu), want))


@pytest.mark.parametrize("mean", [1e-3, 1e-2])
@pytest.mark.parametrize("packed", [False, True])
def test_slow_states(kda, mean, packed):
    """1024 tokens that only decay.  Each rounds its decay and its product by at most 2^-24,
    uncorrelated (a root mean square of 2^-24 sqrt(2 / 3) for both: 1.6e-6 over all),
    and the exponential's error, at most 3e-8 on average, is made up for to 1e-8."""
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.rand(s, generator=gen)  # noqa: E731
    T, dim, S = 1024, 96, 16
    dt, A, init = mean * (0.5 + rnd(1, T, dim)), -(0.7 + 0.6 * rnd(dim, S)), 1 + rnd(1, dim, S)
    zero = torch.zeros(1, T, dim, dtype=BF16, device="cuda")
    cu = torch.tensor([0, T], device="cuda") if packed else None
    for on in (False, True):
        kda.set_segments(on, 0)
        out, fin = kda.ssm_prefill(zero, dt.cuda(), A.cuda(), zero[:, :, :S, None].transpose(2, 3).contiguous(),
                                   zero[:, :, :S, None].transpose(2, 3).contiguous(), init_state=init.cuda(),
                                   cu_seqlens=cu, dt_softplus=False)
        want = init.double() * torch.exp(dt.double().sum(1)[..., None] * A.double())
        off = fin.cpu().double() / want - 1
        assert off.pow(2).mean().sqrt() < 1.6e-6 + 1e-8 * T


@pytest.mark.parametrize("S", [16, 32, 64, 5])
@pytest.mark.parametrize("T,dim", [(1000, 40), (1000, 6000)])
def test_steps_of_zero(kda, T, dim, S):
    """Tokens without a step leave the states as they are, bit for bit, and so do rates of
    zero those that get nothing added."""
    d = draw((1, T), dim, S, 3, bias=False, init=1)
    d["dt"].zero_()
    for on, chunks in ((False, 0), (True, 0), (True, 4)):
        kda.set_segments(on, chunks)
        out, fin = kda.ssm_prefill(**on_gpu(d), dt_softplus=False)
        assert torch.equal(fin.cpu(), d["init_state"])
    d["dt_bias"] = torch.full((dim,), -200.0)
    assert torch.equal(kda.ssm_prefill(**on_gpu(d))[1].cpu(), d["init_state"])
    d["dt_bias"] = torch.full((dim,), 1.0)
    d["A"].zero_()
    d["x"].zero_()
    assert torch.equal(kda.ssm_prefill(**on_gpu(d))[1].cpu(), d["init_state"])


# ------------------------------------------------------------- single tokens

def check_step(kda, d, slots, status=0, softplus=True):
    """d["init_state"] is the pool."""
    dev = on_gpu(d)
    pool = dev.pop("init_state")
    N = d["x"].shape[0]
    at = list(range(N)) if slots is None else slots
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    out = kda.ssm_decode(**dev, state=pool, slots=sl, dt_softplus=softplus)
    torch.cuda.synchronize()
    assert kda.device_status() == status
    have = len(d["init_state"])
    rows = [i for i in range(N) if 0 <= at[i] < have]
    used = [at[i] for i in rows]
    if rows:
        one = {key: t[rows][:, None] if key in ("x", "dt", "B", "C", "z") and t is not None else t for key, t in d.items()}
        one["init_state"] = d["init_state"][used]
        o, f, oe, fe = want_of(one, softplus=softplus, cut=0.0)
        ref.assert_close(out[rows], o[:, 0], oe[:, 0] + scan.rounded(o[:, 0], BF16), "out")
        ref.assert_close(pool[used], f, fe + scan.rounded(f, pool.dtype), "state")
    rest = [p for p in range(have) if p not in used]
    assert torch.equal(pool[rest].cpu(), d["init_state"][rest])
    assert not out[[i for i in range(N) if i not in rows]].any()


@pytest.mark.parametrize("N,dim", [(1, 1), (1, 768), (3, 40), (7, 33), (30, 128), (700, 257)])
@pytest.mark.parametrize("S", [1, 5, 16, 17, 32, 64])
@pytest.mark.parametrize("state", [F32, BF16])
def test_step(kda, N, dim, S, state):
    gen = torch.Generator().manual_seed(N)
    slots = torch.randperm(N + 2, generator=gen)[:N].tolist()
    check_step(kda, draw((N,), dim, S, N * dim + S, init=N + 2, state=state), slots)
    if N < 700:
        check_step(kda, draw((N,), dim, S, N + S, dt=F32, bc=F32, z=False, D=False, bias=False, init=N + 2, state=state,
                             part=3), slots)


@pytest.mark.parametrize("dim,G", [(64, 2), (72, 2), (30, 5)])
def test_step_groups(kda, dim, G):
    check_step(kda, draw((9,), dim, 16, dim, G=G, init=9), None)


@pytest.mark.parametrize("S", [4, 8, 12, 16, 20, 48])
@pytest.mark.parametrize("dt,bc", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
def test_step_types(kda, S, dt, bc):
    for state in (F32, BF16):
        check_step(kda, draw((6,), 36, S, S, G=2, dt=dt, bc=bc, init=8, state=state), [7, -1, 0, 3, 1, 5])


@pytest.mark.parametrize("N", [4, 2500])
def test_step_padding_and_slots(kda, N):
    check_step(kda, draw((N,), 40, 16, 1, init=N), None)
    check_step(kda, draw((N,), 40, 16, 2, init=N + 1), [-1, 2, -7] + [N - i for i in range(N - 3)])
    check_step(kda, draw((N,), 40, 16, 3, init=1), [-1] * N)
    check_step(kda, draw((N,), 40, 16, 4, init=N), [N, 2 ** 31 - 1, 0] + list(range(3, N)), status=8)
    dev = on_gpu(draw((0,), 40, 16, 5))
    dev.pop("init_state")
    pool = torch.ones(2, 40, 16, device="cuda")
    assert kda.ssm_decode(**dev, state=pool).shape == (0, 40) and (pool == 1).all()


def test_step_no_softplus(kda):
    d = draw((5,), 40, 16, 6, init=5, bias=False)
    d["dt"] = d["dt"].abs()
    check_step(kda, d, None, softplus=False)


def test_prompt_then_tokens(kda):
    """A prompt, then single tokens, against the longer prompt."""
    T, more = 133, 6
    d = draw((3, T + more), 72, 16, 12, G=2)
    dev = on_gpu(d)
    dev.pop("init_state")
    o, f, oe, fe = want_of(d)
    per_token = ("x", "dt", "B", "C", "z")
    part = lambda s: {key: t[:, s] if key in per_token else t for key, t in dev.items()}  # noqa: E731
    _, state = kda.ssm_prefill(**{key: t.contiguous() for key, t in part(slice(0, T)).items()})
    for t in range(T, T + more):
        out = kda.ssm_decode(**part(t), state=state)
        ref.assert_close(out, o[:, t], oe[:, t] + scan.rounded(o[:, t], BF16), "token %d" % t)
    ref.assert_close(state, f, fe, "state")


def test_far_slots(kda):
    """States whose offsets pass 32 bits."""
    dim, S, pool = 4096, 64, 8300
    d = draw((2,), dim, S, 13, init=2)
    dev = on_gpu(d)
    init = dev.pop("init_state")
    state = torch.empty(pool, dim, S, device="cuda")
    state[8299], state[3] = init[0], init[1]
    slots = torch.tensor([8299, 3], dtype=torch.int32, device="cuda")
    out = kda.ssm_decode(**dev, state=state, slots=slots)
    want = kda.ssm_decode(**dev, state=init)
    assert torch.equal(out, want) and torch.equal(state[8299], init[0]) and torch.equal(state[3], init[1])


@pytest.mark.parametrize("chunks", [0, 2])
def test_graphs_and_streams(kda, chunks):
    kda.set_segments(True, chunks)
    dev = on_gpu(draw((1, 200), 64, 16, 14, init=2))
    init = dev.pop("init_state")
    cu = torch.tensor([0, 77, 200], device="cuda")
    want = kda.ssm_prefill(**dev, init_state=init, cu_seqlens=cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kda.ssm_prefill(**dev, init_state=init, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, state = torch.empty_like(want[0]), init.clone()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for graph in (first, second):   # each advances the states in place
        with torch.cuda.graph(graph):
            kda.ssm_prefill(**dev, init_state=state, cu_seqlens=cu, out=out, final_state=state)
    state.copy_(init)
    for graph in (first, second, first):
        graph.replay()
    torch.cuda.synchronize()
    s = init
    for _ in range(3):
        y, s = kda.ssm_prefill(**dev, init_state=s, cu_seqlens=cu)
    assert torch.equal(out, y) and torch.equal(state, s)
