"""kda_gated_norm and kda_residual_norm against their formulas in 64 bits.

Bounds: FP32 arithmetic with sums over a row (relative error below 2^-14 for
rows of up to 32,768 elements, whose squares are all positive), then one
rounding to the output's type.
"""

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

D = 128
TYPES = [torch.float32, torch.bfloat16]
EPS = 1e-6


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return m


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g)


def check_gated(kda, x, w, gate, act, first, eps=EPS):
    out = kda.gated_norm(x.cuda(), w.cuda(), None if gate is None else gate.cuda(), activation=act,
                         gate_first=first, eps=eps)
    want = ref.gated_norm(x, w, gate, act, first, eps)
    ref.assert_close(out, want, (ref.HALF_BF16 + 2.0 ** -14) * want.abs() + 2.0 ** -126, "gated norm")


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 64, 65, 257, 1000])
@pytest.mark.parametrize("wt", TYPES)
def test_gated_rows(kda, rows, wt):
    r = gen(rows)
    check_gated(kda, r(rows, D).bfloat16(), (1 + 0.1 * r(D)).to(wt), r(rows, D).bfloat16(), "sigmoid", False)


@pytest.mark.parametrize("act", ["sigmoid", "silu", "none"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("wt", TYPES)
def test_gated_forms(kda, act, first, wt):
    r = gen(3)
    x, w, z = r(3, 5, 6, D).bfloat16(), r(D).to(wt), (8 * r(3, 5, 6, D)).bfloat16()
    x[0, 0, 0] = 0
    x[1, 1] *= 1e-4
    x[2, 2] *= 1e4
    check_gated(kda, x, w, z, act, first)
    if act == "none":
        check_gated(kda, x, w, None, "silu", first)


def test_gated_not_finite(kda):
    r = gen(4)
    x, w, z = r(9, D).bfloat16(), r(D), r(9, D).bfloat16()
    x[2, 3], x[4, 0] = float("nan"), float("inf")
    z[6, 7] = float("nan")
    out = kda.gated_norm(x.cuda(), w.cuda(), z.cuda()).cpu()
    fine = [0, 1, 3, 5, 7, 8]
    want = ref.gated_norm(x, w, z, "sigmoid", False, EPS)
    ref.assert_close(out[fine], want[fine], (ref.HALF_BF16 + 2.0 ** -14) * want[fine].abs(), "other rows")
    assert out[2].isnan().all() and out[4, 0].isnan() and out[6, 7].isnan()
    assert torch.isfinite(out[6]).sum() == D - 1


def test_gated_in_place(kda):
    r = gen(5)
    x, w, z = r(40, D).bfloat16().cuda(), r(D).cuda(), r(40, D).bfloat16().cuda()
    want = kda.gated_norm(x, w, z)
    y = x.clone()
    assert kda.gated_norm(y, w, z, out=y) is y and torch.equal(y, want)
    y = z.clone()
    kda.gated_norm(x, w, y, out=y)
    assert torch.equal(y, want)
    assert kda.gated_norm(x[:0], w, z[:0]).shape == (0, D)


def check_residual(kda, x, r, w, post=None, gate=None, scale=1.0, eps=EPS):
    dev = [None if t is None else t.cuda() for t in (x, r, w, post, gate)]
    out, res = kda.residual_norm(dev[0], dev[1], dev[2], post_weight=dev[3], gate=dev[4], scale=scale, eps=eps)
    o, n, na = ref.residual_norm(x, r, w, post, gate, scale, eps)
    half = ref.HALF_BF16 if r.dtype == torch.bfloat16 else 0.0
    ref.assert_close(res, n, half * n.abs() + 2.0 ** -14 * na, "residual")
    # out follows r' before its rounding: its error is r's, times weight over rms.
    gain = (o / n).abs().nan_to_num(0.0) if n.numel() else o
    ref.assert_close(out, o, (ref.HALF_BF16 + 2.0 ** -14) * o.abs() + 2.0 ** -14 * na * gain, "out")
    return out, res


@pytest.mark.parametrize("dim", [1, 2, 7, 8, 31, 64, 127, 128, 129, 500, 512, 513, 768, 1000, 1024, 1032, 2048, 4095,
                                 4096, 4097, 4104, 8192, 12288, 12296, 16384, 30001, 32760, 32768])
def test_residual_widths(kda, dim):
    r = gen(dim)
    x, res = r(3, dim).bfloat16(), r(3, dim)
    w, post, gate = (r(dim) for _ in range(3))
    check_residual(kda, x, res, w, post, gate, 0.7)
    check_residual(kda, x, res.bfloat16(), w.bfloat16())


@pytest.mark.parametrize("rt", TYPES)
@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("use_post", [False, True])
@pytest.mark.parametrize("use_gate", [False, True])
@pytest.mark.parametrize("dim", [60, 768])
def test_residual_forms(kda, rt, wt, use_post, use_gate, dim):
    r = gen(7)
    x, res, w = r(4, 5, dim).bfloat16(), r(4, 5, dim).to(rt), r(dim).to(wt)
    x[0, 0] = 0
    res[0, 1] = 0
    check_residual(kda, x, res, w, r(dim).to(wt) if use_post else None, r(dim).to(wt) if use_gate else None, -1.5)


@pytest.mark.parametrize("rows", [1, 5, 300, 5000])
def test_residual_rows(kda, rows):
    r = gen(rows)
    check_residual(kda, r(rows, 136).bfloat16(), r(rows, 136), r(136), r(136), None, 0.5)


@pytest.mark.parametrize("rows,dim", [(304, 1032), (700, 2048), (333, 2056), (500, 4096), (310, 4104), (460, 8192),
                                      (305, 12288), (304, 12296), (310, 16384), (400, 4100), (400, 2047)])
@pytest.mark.parametrize("rt", TYPES)
@pytest.mark.parametrize("wt", TYPES)
def test_residual_many_rows(kda, rows, dim, rt, wt):
    """Enough rows for every SM to walk over several."""
    r = gen(rows + dim)
    x, res, w, post, gate = r(rows, dim).bfloat16(), r(rows, dim).to(rt), r(dim).to(wt), r(dim).to(wt), r(dim).to(wt)
    check_residual(kda, x, res, w, post, gate, 0.7)
    check_residual(kda, x, res, w)
    dev = [t.cuda() for t in (x, res, w)]
    want = kda.residual_norm(*dev)
    got = kda.residual_norm(*dev, out=dev[0], residual_out=dev[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows,dim", [(304, 1025), (333, 1026), (311, 4099), (305, 8191), (306, 12289), (304, 16383),
                                      (310, 12282), (1000, 1), (777, 13), (2049, 63), (513, 64), (300, 65), (300, 72),
                                      (300, 255), (301, 257), (300, 512), (333, 770), (300, 1001), (77, 1023)])
@pytest.mark.parametrize("rt", TYPES)
def test_residual_odd_and_narrow_rows(kda, rows, dim, rt):
    """Rows that start at any element, and several rows a warp; in place too."""
    r = gen(rows + dim)
    wt = rt
    x, res, w, post, gate = r(rows, dim).bfloat16(), r(rows, dim).to(rt), r(dim).to(wt), r(dim).to(wt), r(dim).to(wt)
    want = check_residual(kda, x, res, w, post, gate, 0.7)
    check_residual(kda, x, res, w)
    dev = [t.cuda() for t in (x, res, w, post, gate)]
    got = kda.residual_norm(*dev, scale=0.7, out=dev[0], residual_out=dev[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_residual_zero_rows_and_eps(kda):
    x, r, w = torch.zeros(3, 256).bfloat16(), torch.zeros(3, 256), torch.ones(256)
    out, res = check_residual(kda, x, r, w, w, w)
    assert not out.any() and not res.any()
    out, _ = kda.residual_norm(x.cuda(), r.cuda(), w.cuda(), eps=0.0)
    assert out.isnan().all()              # 0 / 0, as the formula has it
    assert kda.residual_norm(x[:0].cuda(), r[:0].cuda(), w.cuda())[0].shape == (0, 256)


def test_residual_in_place(kda):
    r = gen(8)
    x, res, w = r(9, 264).bfloat16().cuda(), r(9, 264).cuda(), r(264).cuda()
    out, new = kda.residual_norm(x, res, w, post_weight=w)
    y, z = x.clone(), res.clone()
    a, b = kda.residual_norm(y, z, w, post_weight=w, out=y, residual_out=z)
    assert a is y and b is z and torch.equal(y, out) and torch.equal(z, new)


def test_residual_not_finite_rows_stay_apart(kda):
    r = gen(9)
    x, res, w = r(4, 300).bfloat16(), r(4, 300), r(300)
    x[1, 5], res[2, 7] = float("nan"), float("inf")
    out, new = (t.cpu() for t in kda.residual_norm(x.cuda(), res.cuda(), w.cuda()))
    o, n, _ = ref.residual_norm(x, res, w, None, None, 1.0, EPS)
    ref.assert_close(out[[0, 3]], o[[0, 3]], 2 * ref.HALF_BF16 * o[[0, 3]].abs() + 1e-3, "other rows")
    assert out[1].isnan().all() and new[1, 5].isnan() and torch.isfinite(new[1]).sum() == 299
    assert new[2, 7] == float("inf")


def test_graph(kda):
    r = gen(10)
    x, z, w = r(30, D).bfloat16().cuda(), r(30, D).bfloat16().cuda(), r(D).cuda()
    res = r(30, D).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = kda.gated_norm(x, w, z)
        o, n = kda.residual_norm(y, res, w)
    x.copy_(r(30, D))
    graph.replay()
    torch.cuda.synchronize()
    y2 = kda.gated_norm(x, w, z)
    o2, n2 = kda.residual_norm(y2, res, w)
    assert torch.equal(y, y2) and torch.equal(o, o2) and torch.equal(n, n2)
