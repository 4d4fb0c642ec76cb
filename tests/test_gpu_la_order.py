"""What a call of kda_la_prefill reads is what the kernels just before it in the
stream wrote: its launches come early (programmatic dependence), so each has to
wait for the end of the one before it ahead of its first read."""

import pytest
import torch

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


@pytest.mark.parametrize("last", ["q", "k", "v", "g", "init"])
@pytest.mark.parametrize("B,T,H,cu", [
    (1, 4100, 4, None),                      # cut by the plan: three kernels
    (2, 8200, 2, None),
    (1, 700, 4, None),                       # not cut
    (1, 4200, 4, [0, 4100, 4200]),           # packed, cut on the device
])
def test_inputs_rewritten_just_before(kda, B, T, H, cu, last):
    """Two sets of inputs in turn in the same buffers, `last` written last; the
    initial and the final states are separate tensors.  Equal bits to calls with
    a pause before and after each, eagerly and in a graph."""
    if cu is None:
        assert (kda.la_plan_segments(B, T, H, False) > 0) == (T > 1000)
    N = B if cu is None else len(cu) - 1
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    sets = [{"q": normal(B, T, H, D).bfloat16(), "k": normal(B, T, H, D).bfloat16(), "v": normal(B, T, H, D).bfloat16(),
             "g": -0.05 * torch.rand((B, T, H), generator=gen, device="cuda"), "init": normal(N, H, D, D)}
            for _ in range(2)]
    at = {key: torch.empty_like(x) for key, x in sets[0].items()}
    cu_t = None if cu is None else torch.tensor(cu, device="cuda")
    order = [key for key in at if key != last] + [last]
    calls = 6

    def chain(pause):
        results = []
        for i in range(calls):
            for key in order:
                at[key].copy_(sets[i % 2][key])
            if pause:
                torch.cuda.synchronize()
            results.append(kda.la_prefill(at["q"], at["k"], at["v"], at["g"], init_state=at["init"], cu_seqlens=cu_t))
            if pause:
                torch.cuda.synchronize()
        return results

    want = chain(True)
    assert not torch.equal(want[0][0], want[1][0]) and not torch.equal(want[0][1], want[1][1])

    def same(got):
        return all(torch.equal(x, y) for pair, other in zip(got, want) for x, y in zip(pair, other))

    for _ in range(3):
        assert same(chain(False))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = chain(False)
    for _ in range(2):
        for pair in got:
            for x in pair:
                x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got)
    assert kda.device_status() == 0


@pytest.mark.parametrize("capture", [False, True])
@pytest.mark.parametrize("T,cu", [(700, None), (4100, None), (900, [0, 500, 500, 900]), (4200, [0, 4100, 4200])])
def test_inputs_from_another_stream(kda, T, cu, capture):
    """A call behind an earlier call of the library and a wait for an event of
    another stream, whose late copies are its inputs: the early launch must not
    pass the event."""
    H, N = 4, 1 if cu is None else len(cu) - 1
    gen = torch.Generator(device="cuda").manual_seed(T)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    src = {"q": normal(1, T, H, D).bfloat16(), "k": normal(1, T, H, D).bfloat16(), "v": normal(1, T, H, D).bfloat16(),
           "g": -0.05 * torch.rand((1, T, H), generator=gen, device="cuda"), "init": normal(N, H, D, D)}
    cu_t = None if cu is None else torch.tensor(cu, device="cuda")
    at = {key: torch.zeros_like(x) for key, x in src.items()}
    big = normal(4096, 4096)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def call(x):
        return kda.la_prefill(x["q"], x["k"], x["v"], x["g"], init_state=x["init"], cu_seqlens=cu_t)

    def run():
        for x in at.values():
            x.zero_()
        call(at)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = big
            for _ in range(12):
                y = y @ big
            for key in at:
                at[key].copy_(src[key])
        call(src)
        torch.cuda.current_stream().wait_stream(side)
        return call(at)

    want = call(src)
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        got = run()
    torch.cuda.synchronize()
    if capture:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            got = run()
    for _ in range(3):
        for x in got:
            x.zero_()
        if capture:
            graph.replay()
        else:
            torch.cuda.synchronize()
            with torch.cuda.stream(main):
                got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert kda.device_status() == 0
