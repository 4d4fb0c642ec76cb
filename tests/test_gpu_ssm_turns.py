"""kda_ssm_prefill where the spans of its chains run in turn, each taking up the state that the one
before it left: against the walk of whole chains bit for bit, against the definition in 64
bits, several calls at once, and the wait between spans where it runs out."""

import ctypes

import pytest
import torch

import ops_reference as ref
import scan_reference as scan
from test_gpu_ssm import BF16, F32, cuts, draw, kda, on_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def in_turn(kda, B, T, dim, G, S, packed):  # noqa: F811
    """Whether such a call's spans run in turn: the scratch it takes with cuts turned off, but for a
    copy of the initial states (where a group is no whole 32 channels) and the offsets' verdict."""
    kda.set_segments(False, 0)
    copy = 0 if dim // G % 32 == 0 else (B * dim * S * 4 + 255) // 256 * 256
    need = kda.ssm_workspace_bytes(B, T, dim, G, S, packed) - copy
    kda.set_segments(True, 0)
    return need > 256 and kda.ssm_plan_segments(B, T, dim, G, S, packed) == 0


def channels(d, lo, hi, G):
    """The call on channels lo .. hi - 1 of one group."""
    dim = d["x"].shape[-1]
    g = lo // (dim // G)
    part = {}
    for key, t in d.items():
        if t is None or key == "cu_seqlens":
            part[key] = t
        elif key in ("B", "C"):
            part[key] = t[:, :, g:g + 1].contiguous()
        elif key in ("A", "D", "dt_bias"):
            part[key] = t[lo:hi].contiguous()
        else:
            part[key] = t[:, lo:hi].contiguous() if key == "init_state" else t[..., lo:hi]
    return part


EDGES = [0, 5, 512, 512, 1024, 1500, 1537, 2100]   # the spans are of 512 tokens
CASES = [  # dim, G, S, B, T, offsets, type of the states, of B and C
    (10240, 1, 16, 1, 2048, None, F32, BF16),
    (5376, 1, 16, 3, 1100, None, F32, BF16),
    (7680, 1, 16, 2, 1500, None, BF16, F32),
    (10240, 1, 16, 1, 2100, EDGES, F32, BF16),
    (10240, 1, 16, 1, 2100, [0, 0, 1, 2099, 2100, 2100], BF16, BF16),
    (15360, 2, 12, 1, 1100, None, F32, BF16),
    (10176, 2, 5, 1, 2048, None, F32, BF16),
    (5376, 1, 32, 2, 1500, None, F32, BF16),
    (10240, 1, 32, 1, 1500, [0, 512, 513, 1500], F32, F32),
    (10000, 2, 32, 1, 1500, None, BF16, BF16),
    (5632, 1, 64, 1, 1500, None, F32, F32),
    (2560, 1, 64, 2, 1100, None, F32, BF16),
    (5632, 1, 64, 1, 2100, EDGES, F32, BF16),
]


@pytest.mark.parametrize("dim,G,S,B,T,cu,state,bc", CASES)
def test_in_turn(kda, dim, G, S, B, T, cu, state, bc):  # noqa: F811
    n = B if cu is None else len(cu) - 1
    assert in_turn(kda, n, T, dim, G, S, cu is not None)
    host = draw((B, T), dim, S, dim + S, G=G, bc=bc, init=n, state=state)
    d = on_gpu(host)
    if cu is not None:
        d["cu_seqlens"] = torch.tensor(cu, device="cuda")
    out, fin = kda.ssm_prefill(**d)
    # Whole chains: the same channels a few at a time.
    kda.set_segments(False, 0)
    for g in range(G):
        for lo in range(g * dim // G, (g + 1) * dim // G, 1000):
            hi = min((g + 1) * dim // G, lo + 1000)
            got = kda.ssm_prefill(**channels(d, lo, hi, G))
            assert torch.equal(got[0], out[..., lo:hi]) and torch.equal(got[1], fin[:, lo:hi])
    kda.set_segments(True, 0)
    # The definition, on the first and the last channels.
    for lo, hi in ((0, 6), (dim - 6, dim)):
        p = channels({**host, "cu_seqlens": None}, lo, hi, G)
        o, f, oe, fe = scan.scan(p["x"], p["dt"], p["A"], p["B"], p["C"], p["D"], p["z"], p["dt_bias"], True,
                                 p["init_state"], cu, cut=0.0)
        ref.assert_close(out[..., lo:hi], o, oe + scan.rounded(o, BF16), "out")
        ref.assert_close(fin[:, lo:hi], f, fe + scan.rounded(f, state), "final")
    # In place, captured and replayed.
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        kept, again = d["init_state"].clone(), torch.empty_like(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            kda.ssm_prefill(**d, out=again, final_state=d["init_state"])
        for _ in range(3):
            d["init_state"].copy_(kept)
            again.zero_()
            graph.replay()
            stream.synchronize()
            assert torch.equal(again, out) and torch.equal(d["init_state"], fin)
    assert kda.device_status() == 0


def test_calls_in_turn_at_once(kda):  # noqa: F811
    """Three such calls on three streams at the same time, two of them captured graphs."""
    shapes = [(1, 2048, 10240, 16), (2, 1500, 7680, 16), (1, 1500, 5632, 64)]
    assert all(in_turn(kda, B, T, dim, 1, S, False) for B, T, dim, S in shapes)
    calls = [on_gpu(draw((B, T), dim, S, dim, init=B)) for B, T, dim, S in shapes]
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


@pytest.mark.parametrize("there", [True, False])
def test_span_wait_runs_out(there):
    """A span whose predecessor's flag is set takes up its state; one whose flag nobody sets waits for the
    bound, which the test library cuts to 10^5 cycles, reports that and ends."""
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    lib = ctypes.CDLL(build.build_test_hooks())
    lib.kda_test_span_wait.argtypes = [ctypes.c_void_p] * 10
    lib.kda_test_span_wait.restype = ctypes.c_int
    d = draw((1, 64), 32, 16, 1, z=False, D=False, bias=False, init=1)
    d["dt"] = d["dt"] - 2
    dev = on_gpu(d)
    out = torch.full((64, 32), 3.0, dtype=BF16, device="cuda")
    states = torch.zeros(2, 32, 16, device="cuda")
    states[0] = dev["init_state"][0]
    relay = torch.tensor([1, int(there), 0], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rc = lib.kda_test_span_wait(*(dev[key].data_ptr() for key in ("x", "dt", "A", "B", "C")), out.data_ptr(),
                                states.data_ptr(), relay.data_ptr(), status.data_ptr(),
                                torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert status.item() == (0 if there else 2)   # KDA_DEV_PIPE_TIMEOUT
    assert relay.tolist() == [2, int(there), 1]
    assert (out[:32] == 3).all()
    half = {key: t[:, 32:] if key in ("x", "dt", "B", "C") else t for key, t in d.items()}
    o, f, oe, fe = scan.scan(half["x"], half["dt"], half["A"], half["B"], half["C"], init=half["init_state"], cut=0.0)
    ref.assert_close(out[None, 32:], o, oe + scan.rounded(o, BF16), "out")
    ref.assert_close(states[1:], f, fe, "state")
