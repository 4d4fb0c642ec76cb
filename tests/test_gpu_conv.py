"""kda_conv_prefill and kda_conv_decode against their definition in 64 bits;
bounds as scan_reference.py derives them, and out's one rounding to BF16.
States are inputs as they are: equal bits."""

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


def draw(lead, D, W, seed, dtype=F32, bias=True, init=None, before=0, after=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    wide = rnd(*lead, before + D + after).bfloat16()
    return {"x": wide[..., before:before + D], "wide": wide, "at": before,
            "w": (0.5 * rnd(D, W)).to(dtype), "bias": rnd(D).to(dtype) if bias else None,
            "init": rnd(init, W - 1, D).bfloat16() if init else None}


def on_gpu(d):
    D = d["x"].shape[-1]
    x = d["wide"].cuda()[..., d["at"]:d["at"] + D]
    return x, *(None if d[key] is None else d[key].cuda() for key in ("w", "bias", "init"))


def check(kda, d, cu=None, act="silu", status=0, **kw):
    x, w, bias, init = on_gpu(d)
    cu_dev = None if cu is None else torch.tensor(cu, device="cuda")
    out, fin = kda.conv_prefill(x, w, bias, init, cu_dev, activation=act, **kw)
    torch.cuda.synchronize()
    assert kda.device_status() == status
    want, final, off = scan.conv(d["x"], d["w"], d["bias"], d["init"], cu, act)
    ref.assert_close(out, want, off + scan.rounded(want, BF16), "out")
    assert torch.equal(fin.cpu(), final.bfloat16())
    return out, fin


@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (1, 2, 3), (2, 3, 64), (3, 5, 10), (1, 33, 768), (2, 130, 257), (1, 1000, 48)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fixed(kda, B, T, D, W, dtype):
    check(kda, draw((B, T), D, W, T * D, dtype))
    check(kda, draw((B, T), D, W, T * D + 1, dtype, bias=False, init=B), act="none")


@pytest.mark.parametrize("lengths", [[5], [0, 7], [1] * 9, [3, 0, 0, 40, 2, 129, 0], [64, 64, 64], [31, 33, 1, 95], [0, 0, 3]])
@pytest.mark.parametrize("D,W", [(24, 4), (10, 3), (7, 4), (768, 2)])
def test_packed(kda, lengths, D, W):
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    for init in (None, len(lengths)):
        check(kda, draw((1, cu[-1]), D, W, cu[-1] + D, init=init), cu)


@pytest.mark.parametrize("D,before,after", [(16, 16, 0), (16, 8, 24), (16, 3, 5), (16, 2, 4), (5, 1, 1)])
def test_part_of_wider_rows(kda, D, before, after):
    check(kda, draw((2, 70), D, 4, 3, before=before, after=after, init=2))
    check(kda, draw((1, 70), D, 3, 4, before=before, after=after, init=3), [0, 30, 30, 70])


def test_no_tokens(kda):
    d = draw((2, 0), 8, 4, 5, init=2)
    _, fin = check(kda, d)
    d = draw((1, 0), 8, 4, 5, init=3)
    check(kda, d, [0, 0, 0, 0])
    d["init"] = None
    _, fin = check(kda, d, [0, 0, 0])
    assert not fin.any()
    x, w, bias, _ = on_gpu(d)
    out, fin = kda.conv_prefill(x, w, bias, output_final_state=False)
    assert fin is None and out.shape == (1, 0, 8)


@pytest.mark.parametrize("cu", [[0, 5, 4, 9], [1, 5, 9], [0, 5, 8], [0, 12, 9], [-1, 4, 9]])
def test_bad_offsets(kda, cu):
    """The host cannot see them: nothing is written."""
    x, w, bias, _ = on_gpu(draw((1, 9), 16, 4, 6))
    out = torch.full((1, 9, 16), 3.0, dtype=BF16, device="cuda")
    fin = torch.full((len(cu) - 1, 3, 16), 3.0, dtype=BF16, device="cuda")
    kda.conv_prefill(x, w, bias, cu_seqlens=torch.tensor(cu, device="cuda"), out=out, final_state=fin)
    torch.cuda.synchronize()
    assert kda.device_status() == 1
    assert (out == 3).all() and (fin == 3).all()


@pytest.mark.parametrize("bad", [False, True])
def test_many_sequences(kda, bad):
    """More offsets than a CTA checks by itself."""
    gen = torch.Generator().manual_seed(7)
    lengths = torch.randint(0, 4, (1500,), generator=gen).tolist()
    cu = [0] + torch.tensor(lengths).cumsum(0).tolist()
    d = draw((1, cu[-1]), 8, 4, 8, init=1500)
    if not bad:
        check(kda, d, cu)
        return
    x, w, bias, init = on_gpu(d)
    cu[700] = cu[701] + 1
    out = torch.full(x.shape, 3.0, dtype=BF16, device="cuda")
    kda.conv_prefill(x, w, bias, init, torch.tensor(cu, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert kda.device_status() == 1 and (out == 3).all()


def test_states_in_place(kda):
    for lead, cu in (((2, 100), None), ((2, 1), None), ((1, 100), [0, 2, 60, 60, 100])):
        n = lead[0] if cu is None else len(cu) - 1
        d = draw(lead, 40, 4, 9, init=n)
        x, w, bias, init = on_gpu(d)
        cu_dev = None if cu is None else torch.tensor(cu, device="cuda")
        want = kda.conv_prefill(x, w, bias, init, cu_dev)
        got = kda.conv_prefill(x, w, bias, init, cu_dev, final_state=init)
        assert got[1] is init and all(torch.equal(a, b) for a, b in zip(got, want))


def test_prompt_in_parts(kda):
    """A prompt in two calls gives the bits of one."""
    x, w, bias, _ = on_gpu(draw((1, 333), 64, 4, 10))
    whole, last = kda.conv_prefill(x, w, bias)
    for at in (1, 2, 3, 100, 332):
        a, s = kda.conv_prefill(x[:, :at], w, bias)
        b, s = kda.conv_prefill(x[:, at:], w, bias, s)
        assert torch.equal(torch.cat([a, b], 1), whole) and torch.equal(s, last)


def test_far_rows(kda):
    """Rows whose offsets pass 32 bits."""
    d = draw((1, 40), 16, 4, 11)
    wide = torch.empty(1, 40, 1 << 26, dtype=BF16, device="cuda")
    x = wide[..., 64:80]
    x.copy_(d["x"].cuda())
    _, w, bias, _ = on_gpu(d)
    got = kda.conv_prefill(x, w, bias)
    want = kda.conv_prefill(d["x"].cuda().contiguous(), w, bias)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(kda, value):
    d = draw((2, 50), 24, 4, 12, init=2)
    d["x"][0, 20, 5] = value
    d["init"][1, 1, 3] = value
    check(kda, d, act="none")
    x, w, bias, init = on_gpu(d)
    out, _ = kda.conv_prefill(x, w, bias, init)
    fine = torch.isfinite(out.float()).cpu()
    assert not fine[0, 20:24, 5].all()
    fine[0, 20:24, 5] = True
    fine[1, :2, 3] = True
    assert fine.all()


# ------------------------------------------------------------- single tokens

def check_step(kda, d, slots, act="silu", status=0):
    """d["init"] is the pool."""
    x, w, bias, pool = on_gpu(d)
    N, W = d["x"].shape[0], d["w"].shape[1]
    at = list(range(N)) if slots is None else slots
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    out = kda.conv_decode(x, w, pool, bias, sl, act)
    torch.cuda.synchronize()
    assert kda.device_status() == status
    rows = [i for i in range(N) if 0 <= at[i] < len(d["init"])]
    used = [at[i] for i in rows]
    new = d["init"].clone()
    if rows:
        want, final, off = scan.conv(d["x"][rows][:, None], d["w"], d["bias"], d["init"][used], act=act)
        ref.assert_close(out[rows], want[:, 0], off[:, 0] + scan.rounded(want[:, 0], BF16), "out")
        new[used] = final.bfloat16()
    assert torch.equal(pool.cpu(), new)
    assert W - 1 == pool.shape[1] and not out[[i for i in range(N) if i not in rows]].any()


@pytest.mark.parametrize("N,D", [(1, 8), (1, 2304), (3, 10), (7, 5), (30, 768), (600, 2304), (601, 1030)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step(kda, N, D, W, dtype):
    gen = torch.Generator().manual_seed(N)
    d = draw((N,), D, W, N * D, dtype, bias=W != 3, init=N + 2, before=D if W == 4 else 0)
    check_step(kda, d, torch.randperm(N + 2, generator=gen)[:N].tolist(), "none" if W == 2 else "silu")


@pytest.mark.parametrize("N", [4, 700])
def test_step_padding_and_slots(kda, N):
    D = 16 if N == 4 else 1024
    check_step(kda, draw((N,), D, 4, 1, init=N), None)
    check_step(kda, draw((N,), D, 4, 2, init=N + 1), [-1, 2, -7] + [N - i for i in range(N - 3)])
    check_step(kda, draw((N,), D, 4, 3, init=1), [-1] * N)
    check_step(kda, draw((N,), D, 4, 4, init=N), [N, 2 ** 31 - 1, 0] + list(range(3, N)), status=8)
    x, w, bias, _ = on_gpu(draw((0,), D, 4, 5))
    pool = torch.ones(2, 3, D, dtype=BF16, device="cuda")
    assert kda.conv_decode(x, w, pool, bias).shape == (0, D) and (pool == 1).all()


def test_prompt_then_tokens(kda):
    """Tokens one by one give the bits of the whole prompt."""
    x, w, bias, _ = on_gpu(draw((3, 90), 40, 4, 13))
    whole, last = kda.conv_prefill(x, w, bias)
    _, pool = kda.conv_prefill(x[:, :70].contiguous(), w, bias)
    for t in range(70, 90):
        assert torch.equal(kda.conv_decode(x[:, t], w, pool, bias), whole[:, t])
    assert torch.equal(pool, last)


def test_far_slots(kda):
    """States whose offsets pass 32 bits."""
    D, pool = 1 << 20, 720
    state = torch.empty(pool, 3, D, dtype=BF16, device="cuda")
    d = draw((2,), D, 4, 14, bias=False, init=2)
    x, w, _, init = on_gpu(d)
    state[719], state[3] = init[0], init[1]
    slots = torch.tensor([719, 3], dtype=torch.int32, device="cuda")
    out = kda.conv_decode(x, w, state, slots=slots)
    want = kda.conv_decode(x, w, init)
    assert torch.equal(out, want) and torch.equal(state[719], init[0]) and torch.equal(state[3], init[1])


def test_graphs_and_streams(kda):
    d = draw((1, 100), 64, 4, 15, init=2)
    x, w, bias, init = on_gpu(d)
    cu = torch.tensor([0, 37, 100], device="cuda")
    want = kda.conv_prefill(x, w, bias, init, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kda.conv_prefill(x, w, bias, init, cu, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out, state = torch.empty_like(want[0]), init.clone()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for graph in (first, second):   # each advances the states in place
        with torch.cuda.graph(graph):
            kda.conv_prefill(x, w, bias, state, cu, out=out, final_state=state)
    state.copy_(init)
    for graph in (first, second, first):
        graph.replay()
    torch.cuda.synchronize()
    s = init
    for _ in range(3):
        y, s = kda.conv_prefill(x, w, bias, s, cu)
    assert torch.equal(out, y) and torch.equal(state, s)
