"""kda_la_prefill against the recurrence token by token in 64 bits.

Bounds.  out is BF16 (one rounding of at most 2^-8 of the value) and its
products take the scores, the scaled queries and the incoming states in BF16:
at most two such roundings in any term, each 2^-8 of the term's magnitude.
The state is FP32: each chunk's keys enter as two BF16 parts (2^-16 of a
term's magnitude), FP32 sums of up to 128 + chunks terms, and exponents whose
sums are off by 2^-24 of at most 128 terms: together under 2^-14 of the
magnitude; a BF16 state adds one rounding.  Sums of squares are also compared:
the bounds above are reached only where every rounding has the same sign.
"""

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


def inputs(B, T, H, Hk=None, seed=0, g="token", init=None, low=-0.5):
    gen = torch.Generator().manual_seed(seed)
    Hk = Hk or H
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d = {"q": rnd(B, T, Hk, D).bfloat16(), "k": rnd(B, T, Hk, D).bfloat16(), "v": rnd(B, T, H, D).bfloat16(),
         "g": low * (torch.rand((H,) if g == "head" else (B, T, H), generator=gen))}
    return d, rnd


def run(kda, d, init=None, cu=None, **kw):
    dev = {key: x.cuda() for key, x in d.items()}
    out, fin = kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"],
                              init_state=None if init is None else init.cuda(),
                              cu_seqlens=None if cu is None else torch.tensor(cu, device="cuda"), **kw)
    torch.cuda.synchronize()
    assert kda.device_status() == 0
    return out.cpu(), fin.cpu()


def check(kda, d, init=None, cu=None, rel=True, **kw):
    out, fin = run(kda, d, init, cu, **kw)
    o, f, oa, fa = ref.la_tokens(d["q"], d["k"], d["v"], d["g"], init, cu, kw.get("scale", ref.SCALE))
    ref.assert_close(out, o, ref.HALF_BF16 * o.abs() + 2.1 * ref.HALF_BF16 * oa, "out")
    half = ref.HALF_BF16 if fin.dtype == torch.bfloat16 else 0.0
    ref.assert_close(fin, f, 2.0 ** -14 * fa + half * f.abs(), "final state")
    if rel and o.numel() and torch.isfinite(o).all():
        assert (out.double() - o).norm() <= 1e-2 * o.norm()
        if f.norm() > 0:
            assert (fin.double() - f).norm() <= (1e-2 if half else 2e-5) * f.norm()


@pytest.mark.parametrize("T", [1, 2, 15, 16, 31, 64, 127, 128, 129, 200, 255, 256, 257, 385, 700])
def test_lengths(kda, T):
    d, rnd = inputs(1, T, 2, seed=T)
    check(kda, d, init=rnd(1, 2, D, D))


@pytest.mark.parametrize("B,T,H,Hk", [(3, 77, 6, 6), (2, 130, 12, 4), (5, 33, 8, 1), (1, 300, 3, 3)])
@pytest.mark.parametrize("g", ["token", "head"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_heads_decays_and_states(kda, B, T, H, Hk, g, dtype):
    d, rnd = inputs(B, T, H, Hk, seed=B * T, g=g)
    check(kda, d, init=rnd(B, H, D, D).to(dtype))
    check(kda, d, state_dtype=dtype)


@pytest.mark.parametrize("lengths", [[5], [0, 7, 0, 128, 1], [129, 3, 250, 64, 0], [1] * 9, [0, 0], [300, 128, 17]])
def test_packed(kda, lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    d, rnd = inputs(1, cu[-1], 4, 2, seed=sum(lengths))
    check(kda, d, init=rnd(len(lengths), 4, D, D), cu=cu)
    check(kda, d, cu=cu, state_dtype=torch.bfloat16)


@pytest.mark.parametrize("seg", [8, 24])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("init", [False, True])
def test_segments(kda, seg, packed, init):
    """Forced segments: their lengths are whole 128-token chunks."""
    kda.set_segments(True, seg)
    try:
        if packed:
            cu = [0, 300, 300, 1100, 1101, 1485]
            d, rnd = inputs(1, cu[-1], 2, 1, seed=5, low=-0.05)
            N = len(cu) - 1
        else:
            cu, N = None, 2
            d, rnd = inputs(2, 1000, 2, 1, seed=6, low=-0.05)
        st = rnd(N, 2, D, D) if init else None
        check(kda, d, init=st, cu=cu)
        check(kda, d, init=None if st is None else st.bfloat16(), cu=cu)
    finally:
        kda.set_segments(True, 0)


def test_planned_segments(kda):
    """A shape that the plan itself cuts agrees with the uncut chain."""
    assert kda.la_plan_segments(1, 4100, 2, False) > 1
    d, rnd = inputs(1, 4100, 2, seed=9, low=-0.02)
    init = rnd(1, 2, D, D)
    out, fin = run(kda, d, init)
    kda.set_segments(False)
    try:
        assert kda.la_plan_segments(1, 4100, 2, False) == 0
        out2, fin2 = run(kda, d, init)
    finally:
        kda.set_segments(True, 0)
    o, f, oa, fa = ref.la_tokens(d["q"], d["k"], d["v"], d["g"], init)
    for x, y in ((out, fin), (out2, fin2)):
        ref.assert_close(x, o, ref.HALF_BF16 * o.abs() + 2.1 * ref.HALF_BF16 * oa, "out")
        ref.assert_close(y, f, 2.0 ** -14 * fa, "final state")


@pytest.mark.parametrize("seg", [0, 8])
@pytest.mark.parametrize("value", [-5.0, -40.0, -200.0, -1e30, float("-inf"), 0.0, -0.0])
def test_decay_extremes(kda, value, seg):
    d, rnd = inputs(1, 390, 2, seed=11)
    d["g"][0, :, 0] = value                       # every token of a head
    d["g"][0, 130::37, 1] = value                 # single tokens of another
    kda.set_segments(True, seg)
    try:
        check(kda, d, init=rnd(1, 2, D, D))
    finally:
        kda.set_segments(True, 0)


@pytest.mark.parametrize("size", [1e-6, 1e4])
@pytest.mark.parametrize("low", [-0.02, -0.6, -1.2, -20.0])
def test_large_and_small_values(kda, size, low):
    """Decays of a chunk from next to none to many powers of two: the bounds are
    relative to the values."""
    d, rnd = inputs(1, 390, 3, 1, seed=53, low=low)
    d["g"][:, :, 2] = low                          # the same at every token
    for key in ("q", "k", "v"):
        d[key] = (d[key].float() * size).bfloat16()
    check(kda, d, init=rnd(1, 3, D, D) * size * size)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "g"])
def test_not_finite(kda, where, bad):
    """A bad token reaches neither earlier tokens, nor other heads, nor other
    sequences; the later ones of its own sequence and head that the recurrence
    spoils are not finite either."""
    if where == "g" and bad == float("-inf"):
        pytest.skip("-inf is a decay: it forgets the state")
    cu = [0, 100, 260, 270, 400]
    d, rnd = inputs(1, 400, 2, seed=13)
    clean, cfin = run(kda, d, cu=cu)
    t = 170                                       # token 70 of the second sequence
    if where == "g":
        d["g"][0, t, 1] = bad
    else:
        d[where][0, t, 1, 5] = bad
    out, fin = run(kda, d, cu=cu)
    assert torch.equal(out[0, :, 0], clean[0, :, 0])
    assert torch.equal(out[0, :t, 1], clean[0, :t, 1])
    assert torch.equal(out[0, 260:, 1], clean[0, 260:, 1])
    assert torch.equal(fin[:, 0], cfin[:, 0]) and torch.equal(fin[[0, 2, 3], 1], cfin[[0, 2, 3], 1])
    o, f, _, _ = ref.la_tokens(d["q"], d["k"], d["v"], d["g"], None, cu)
    assert torch.equal(torch.isfinite(out[0, :, 1]), torch.isfinite(o[0, :, 1]))
    assert torch.equal(torch.isfinite(fin[:, 1]), torch.isfinite(f[:, 1]))


def test_garbage_behind_sequences_ends(kda):
    """Padding tokens after a row's last token may hold anything."""
    d, _ = inputs(2, 150, 2, seed=17)
    clean, _ = run(kda, d)
    for key in ("q", "k", "v", "g"):
        d[key][:, 141:] = float("nan")
    out, _ = run(kda, d)
    assert torch.equal(out[:, :141], clean[:, :141])


def test_state_in_place_and_no_final(kda):
    d, rnd = inputs(2, 140, 2, seed=19)
    init = rnd(2, 2, D, D)
    out, fin = run(kda, d, init)
    dev = {key: x.cuda() for key, x in d.items()}
    st = init.cuda()
    o2, f2 = kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], init_state=st, final_state=st)
    assert f2 is st and torch.equal(st.cpu(), fin) and torch.equal(o2.cpu(), out)
    o3, f3 = kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], init_state=init.cuda(), output_final_state=False)
    assert f3 is None and torch.equal(o3.cpu(), out)


@pytest.mark.parametrize("seg", [0, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cu", [None, [0, 40, 40, 5040, 5110]])
def test_state_in_place_with_segments(kda, cu, dtype, seg):
    T = 5110 if cu else 4100
    d, rnd = inputs(1, T, 4, 2, seed=47, low=-0.02)
    init = rnd(len(cu) - 1 if cu else 1, 4, D, D).to(dtype)
    dev = {key: x.cuda() for key, x in d.items()}
    kda.set_segments(True, seg)
    try:
        out, fin = run(kda, d, init, cu)
        for _ in range(3):
            st = init.cuda()
            o2, _ = kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], init_state=st, final_state=st,
                                   cu_seqlens=None if cu is None else torch.tensor(cu, device="cuda"))
            assert torch.equal(st.cpu(), fin) and torch.equal(o2.cpu(), out)
    finally:
        kda.set_segments(True, 0)


def test_no_tokens(kda):
    init = torch.randn(2, 3, D, D)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for st in (init, init.bfloat16()):
        out, fin = kda.la_prefill(e(2, 0, 3, D), e(2, 0, 3, D), e(2, 0, 3, D),
                                  torch.empty(2, 0, 3, device="cuda"), init_state=st.cuda())
        assert out.numel() == 0 and torch.equal(fin.cpu(), st)
    _, fin = kda.la_prefill(e(2, 0, 3, D), e(2, 0, 3, D), e(2, 0, 3, D), torch.empty(2, 0, 3, device="cuda"))
    assert not fin.any()


def test_two_halves_give_the_whole(kda):
    d, rnd = inputs(1, 400, 2, seed=23)
    init = rnd(1, 2, D, D)
    o, f, oa, fa = ref.la_tokens(d["q"], d["k"], d["v"], d["g"], init)
    cut = 173
    parts = [{key: x[:, s].contiguous() for key, x in d.items()} for s in (slice(0, cut), slice(cut, None))]
    o1, f1 = run(kda, parts[0], init)
    o2, f2 = run(kda, parts[1], f1)
    ref.assert_close(torch.cat([o1, o2], 1), o, ref.HALF_BF16 * o.abs() + 2.1 * ref.HALF_BF16 * oa, "out")
    ref.assert_close(f2, f, 2.0 ** -13 * fa, "final state")


def test_bad_offsets_touch_nothing(kda):
    d, _ = inputs(1, 50, 2, seed=29)
    dev = {key: x.cuda() for key, x in d.items()}
    for cu in ([0, 30, 20, 50], [0, 20, 49], [1, 20, 50]):
        out = torch.full_like(dev["v"], 7)
        fin = torch.full((len(cu) - 1, 2, D, D), 7.0, device="cuda")
        kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], cu_seqlens=torch.tensor(cu, device="cuda"),
                       out=out, final_state=fin)
        assert kda.device_status() == 1
        assert (out == 7).all() and (fin == 7).all()


@pytest.mark.parametrize("B,T,H,cu", [(1, 700, 2, None), (1, 4100, 2, None), (1, 900, 4, [0, 500, 500, 900])])
def test_graph_and_determinism(kda, B, T, H, cu):
    """A captured call replays on fresh inputs; equal inputs give equal bits."""
    d, _ = inputs(B, T, H, seed=31, low=-0.1)
    dev = {key: x.cuda() for key, x in d.items()}
    cu_t = None if cu is None else torch.tensor(cu, device="cuda")
    out, fin = torch.empty_like(dev["v"]), torch.empty((len(cu) - 1 if cu else B, H, D, D), device="cuda")
    call = lambda: kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], cu_seqlens=cu_t, out=out,  # noqa: E731
                                  final_state=fin)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    fresh, _ = inputs(B, T, H, seed=37, low=-0.1)
    for key in dev:
        dev[key].copy_(fresh[key])
    want = [x.clone() for x in call()]
    for _ in range(3):
        out.fill_(float("nan"))
        fin.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(fin, want[1])
    assert kda.device_status() == 0


def heads(x, hs, Hk, H):
    """The inputs of heads hs alone."""
    ks = [h // (H // Hk) for h in hs]
    return {"q": x["q"][:, :, ks], "k": x["k"][:, :, ks], "v": x["v"][:, :, hs],
            "g": x["g"][hs] if x["g"].dim() == 1 else x["g"][:, :, hs]}


def check_heads(kda, d, init, cu, hs, Hk, H):
    """The whole call, compared on some heads."""
    out, fin = run(kda, d, init, cu)
    sub = heads(d, hs, Hk, H)
    o, f, oa, fa = ref.la_tokens(sub["q"], sub["k"], sub["v"], sub["g"], None if init is None else init[:, hs], cu)
    half = ref.HALF_BF16 if fin.dtype == torch.bfloat16 else 0.0
    ref.assert_close(out[:, :, hs], o, ref.HALF_BF16 * o.abs() + 2.1 * ref.HALF_BF16 * oa, "out")
    ref.assert_close(fin[:, hs], f, 2.0 ** -14 * fa + half * f.abs(), "final state")


def offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", [[40, 0, 5000, 70, 300], [5000], [2500, 1, 2500], [0, 4097, 0]])
def test_packed_cut_on_the_device(kda, lengths, dtype):
    """One long sequence among short ones, few heads: cut by the plan itself."""
    cu = offsets(lengths)
    d, rnd = inputs(1, cu[-1], 2, 1, seed=len(lengths), low=-0.02)
    check(kda, d, init=rnd(len(lengths), 2, D, D).to(dtype), cu=cu)
    check(kda, d, cu=cu, state_dtype=dtype)


@pytest.mark.parametrize("H,Hk", [(8, 8), (96, 32)])
def test_packed_longest_first(kda, H, Hk):
    """More units than SMs: the sequences go by their lengths; zeros and ties."""
    lengths = [(37 * i) % 151 for i in range(40)] + [0, 0, 150, 150] if H == 8 else [700, 0, 20, 900, 20, 600]
    cu = offsets(lengths)
    d, rnd = inputs(1, cu[-1], H, Hk, seed=H, low=-0.05)
    check_heads(kda, d, rnd(len(lengths), H, D, D), cu, [0, 5, H - 1], Hk, H)


@pytest.mark.parametrize("top", [2, 6])
def test_packed_many_sequences(kda, top):
    """More sequences than one block has threads, most of them short or empty."""
    lengths = [(7 * i) % top for i in range(1100)]
    cu = offsets(lengths)
    d, rnd = inputs(1, cu[-1], 2, seed=top)
    check(kda, d, init=rnd(len(lengths), 2, D, D), cu=cu)


@pytest.mark.parametrize("B,T,H,Hk,seg,cu", [
    (2, 900, 12, 4, 24, None),                      # many units: one warp a part of the scan
    (1, 1100, 24, 24, 8, [0, 700, 700, 1100]),
    (1, 4500, 1, 1, 8, None),                       # many segments of few units
    (1, 4500, 2, 1, 8, [0, 4400, 4500]),
])
def test_segment_scans(kda, B, T, H, Hk, seg, cu):
    kda.set_segments(True, seg)
    try:
        d, rnd = inputs(B, T, H, Hk, seed=T, low=-0.03)
        init = rnd(len(cu) - 1 if cu else B, H, D, D)
        hs = sorted({0, H // 2, H - 1})
        check_heads(kda, d, init, cu, hs, Hk, H)
        check_heads(kda, d, init.bfloat16(), cu, hs, Hk, H)
    finally:
        kda.set_segments(True, 0)


@pytest.mark.parametrize("H", [2, 96])
def test_bad_offsets_of_larger_batches_touch_nothing(kda, H):
    d, _ = inputs(1, 2500, H, seed=43)
    dev = {key: x.cuda() for key, x in d.items()}
    many = [min(n, 2500) for n in range(0, 4400, 4)]
    many[600] = many[602] + 1
    for cu in ([0, 1500, 1000, 2500], [0, 1000, 2499], [-1, 1000, 2500], [0, 1 << 40, 2500], many):
        out = torch.full_like(dev["v"], 7)
        fin = torch.full((len(cu) - 1, H, D, D), 7.0, device="cuda")
        kda.la_prefill(dev["q"], dev["k"], dev["v"], dev["g"], cu_seqlens=torch.tensor(cu, device="cuda"),
                       out=out, final_state=fin)
        assert kda.device_status() == 1
        assert (out == 7).all() and (fin == 7).all()


@pytest.mark.parametrize("T,cu", [(77, None), (700, [0, 100, 700]), (4100, None), (4200, [0, 4100, 4200])])
def test_calls_in_a_row(kda, T, cu):
    """Each call reads what the one before it wrote, without a pause between
    them, eagerly and in a graph behind a copy and a fill."""
    d, _ = inputs(1, T, 4, seed=59, low=-0.05)
    dev = {key: x.cuda() for key, x in d.items()}
    cu_t = None if cu is None else torch.tensor(cu, device="cuda")
    st = torch.zeros(1 if cu is None else len(cu) - 1, 4, D, D, device="cuda")
    bufs = [torch.empty_like(dev["v"]) for _ in range(3)]
    src = torch.empty_like(dev["q"])

    def chain(pause):
        src.copy_(dev["q"])
        st.zero_()
        x = src
        for i in range(8):
            out = bufs[i % 3]
            # (Outputs of a size that stays: the scale undoes their growth.)
            kda.la_prefill(x, dev["k"], x, dev["g"], init_state=st, final_state=st, cu_seqlens=cu_t, out=out,
                           scale=2.0 ** -10)
            if pause:
                torch.cuda.synchronize()
            x = out
        return x

    want, state = chain(True).clone(), st.clone()
    assert torch.isfinite(want).all()
    for _ in range(5):
        got = chain(False)
        assert torch.equal(got, want) and torch.equal(st, state)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = chain(False)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(st, state)
    assert kda.device_status() == 0


@pytest.mark.slow
def test_many_heads_long(kda):
    """More chains than SMs, and chunks enough for every buffer to be reused."""
    d, rnd = inputs(2, 1500, 96, 32, seed=41, low=-0.05)
    init = rnd(2, 96, D, D)
    out, fin = run(kda, d, init)
    hs = [0, 37, 95]
    sub = {"q": d["q"][:, :, [h // 3 for h in hs]], "k": d["k"][:, :, [h // 3 for h in hs]],
           "v": d["v"][:, :, hs], "g": d["g"][:, :, hs]}
    o, f, oa, fa = ref.la_tokens(sub["q"], sub["k"], sub["v"], sub["g"], init[:, hs])
    ref.assert_close(out[:, :, hs], o, ref.HALF_BF16 * o.abs() + 2.1 * ref.HALF_BF16 * oa, "out")
    ref.assert_close(fin[:, hs], f, 2.0 ** -14 * fa, "final state")
