"""Refusals of the convolution and the scan (no GPU needed): bad arguments are
turned away on the host, before any CUDA call.  Addresses passed here are never
dereferenced."""

import ctypes

import pytest
import torch

from kimi_delta_attention_kda_gb300 import _lib, build, ops

A, GB = 1 << 20, 1 << 32


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def no_gpu():
    return not torch.cuda.is_available()


def at(i):
    return A + i * GB


def conv(lib, x=at(0), ldx=64, w=at(1), bias=at(2), init=at(3), out=at(4), fin=at(5), B=2, T=16, D=64, W=4, cu=None,
         act=2, flags=0):
    return lib.kda_conv_prefill(x, ldx, w, bias, init, out, fin, B, T, D, W, cu, act, flags, None)


def test_conv_prefill(lib):
    for kw in (dict(flags=2), dict(flags=256), dict(act=1), dict(act=3), dict(act=-1)):
        assert conv(lib, **kw) == -7, kw
    for kw in (dict(B=0), dict(T=-1), dict(D=0), dict(W=1), dict(W=5), dict(ldx=63), dict(ldx=-64), dict(T=1 << 31),
               dict(B=1 << 40), dict(B=1 << 20, T=1 << 20), dict(D=1 << 60), dict(ldx=1 << 60)):
        assert conv(lib, **kw) == -2, kw
    for name in ("x", "w", "out"):
        assert conv(lib, **{name: None}) == -1, name
    for kw in (dict(x=at(0) + 1), dict(w=at(1) + 8), dict(bias=at(2) + 8), dict(init=at(3) + 8), dict(out=at(4) + 8),
               dict(fin=at(5) + 8), dict(cu=at(6) + 4)):
        assert conv(lib, **kw) == -3, kw
    # Rows 1,024 elements apart: x ends 31 such rows and 64 elements behind its start.
    far = dict(ldx=1024, x=at(0))
    for kw in (dict(out=at(0)), dict(out=at(0) + 2 * (31 * 1024 + 48), **far), dict(out=at(1)), dict(out=at(3)),
               dict(fin=at(4)), dict(fin=at(0)), dict(init=at(5), fin=at(5) + 16), dict(fin=at(6), cu=at(6)), dict(out=at(2))):
        assert conv(lib, **kw) == -4, kw
    if no_gpu():
        assert conv(lib) == -5 and conv(lib, init=at(5)) == -5 and conv(lib, x=at(0) + 2) == -5
        assert conv(lib, out=at(0) + 2 * (31 * 1024 + 64), **far) == -5
        assert conv(lib, bias=None, init=None, fin=None, W=2, act=0, flags=8) == -5
        assert conv(lib, x=None, out=None, T=0) == -5 and conv(lib, B=1, T=1, ldx=0) == -5


def conv_step(lib, x=at(0), ldx=64, w=at(1), bias=at(2), state=at(3), slots=at(4), out=at(5), N=2, D=64, W=4, pool=3,
              act=2, flags=0):
    return lib.kda_conv_decode(x, ldx, w, bias, state, slots, out, N, D, W, pool, act, flags, None)


def test_conv_decode(lib):
    for kw in (dict(flags=2), dict(act=1), dict(act=3)):
        assert conv_step(lib, **kw) == -7, kw
    for kw in (dict(N=-1), dict(D=0), dict(W=1), dict(W=5), dict(pool=-1), dict(slots=None, pool=1), dict(ldx=63),
               dict(pool=1 << 60), dict(D=1 << 60), dict(N=1 << 40)):
        assert conv_step(lib, **kw) == -2, kw
    for name in ("x", "w", "out", "state"):
        assert conv_step(lib, **{name: None}) == -1, name
    for kw in (dict(x=at(0) + 1), dict(w=at(1) + 8), dict(bias=at(2) + 8), dict(state=at(3) + 8), dict(out=at(5) + 8),
               dict(slots=at(4) + 2)):
        assert conv_step(lib, **kw) == -3, kw
    for kw in (dict(out=at(0)), dict(out=at(3) + 16), dict(state=at(1)), dict(state=at(4)), dict(out=at(2))):
        assert conv_step(lib, **kw) == -4, kw
    if no_gpu():
        assert conv_step(lib) == -5 and conv_step(lib, slots=None) == -5 and conv_step(lib, pool=0, state=None) == -5


NAMES = "x ldx dt lddt A B ldb C ldc D z ldz bias".split()
READ = dict(x=at(0), ldx=64, dt=at(1), lddt=64, A=at(2), B=at(3), ldb=32, C=at(4), ldc=32, D=at(5), z=at(6), ldz=64, bias=at(7))


def ssm(lib, init=at(8), out=at(9), fin=at(10), n=2, T=16, dim=64, groups=2, S=16, cu=None, flags=256, **kw):
    args = {**READ, **kw}
    return lib.kda_ssm_prefill(*(args[k] for k in NAMES), init, out, fin, n, T, dim, groups, S, cu, flags, None)


def ssm_step(lib, state=at(8), slots=at(10), out=at(9), n=2, dim=64, groups=2, S=16, pool=3, flags=256, **kw):
    args = {**READ, **kw}
    return lib.kda_ssm_decode(*(args[k] for k in NAMES), state, slots, out, n, dim, groups, S, pool, flags, None)


@pytest.mark.parametrize("call", [ssm, ssm_step])
def test_scan(lib, call):
    for flags in (1, 4, 8, 512):
        assert call(lib, flags=flags) == -7
    for kw in (dict(dim=0), dict(groups=0), dict(groups=3), dict(S=0), dict(S=65), dict(n=-1), dict(n=1 << 40),
               dict(dim=1 << 24), dict(ldx=63), dict(lddt=63), dict(ldb=31), dict(ldc=31), dict(ldz=63), dict(ldx=1 << 60)):
        assert call(lib, **kw) == -2, kw
    for name in ("x", "dt", "A", "B", "C", "out"):
        assert call(lib, **{name: None}) == -1, name
    for kw in (dict(x=at(0) + 1), dict(dt=at(1) + 1), dict(dt=at(1) + 2, flags=64), dict(A=at(2) + 8), dict(B=at(3) + 1),
               dict(C=at(4) + 2, flags=128), dict(D=at(5) + 2), dict(z=at(6) + 1), dict(bias=at(7) + 2), dict(out=at(9) + 8)):
        assert call(lib, **kw) == -3, kw
    for i in range(8):
        assert call(lib, out=at(i)) == -4, i
    if no_gpu():
        assert call(lib) == -5 and call(lib, D=None, z=None, ldz=0, bias=None, flags=2 | 64 | 128) == -5
        assert call(lib, x=at(0) + 2, dt=at(1) + 2, B=at(3) + 2, C=at(4) + 2, z=at(6) + 2) == -5


def test_scan_own_arguments(lib):
    assert ssm(lib, n=0) == -2 and ssm(lib, T=-1) == -2 and ssm(lib, T=1 << 31) == -2
    for kw in (dict(init=at(8) + 8), dict(fin=at(10) + 8), dict(cu=at(11) + 4)):
        assert ssm(lib, **kw) == -3, kw
    for kw in (dict(fin=at(9)), dict(fin=at(0)), dict(fin=at(2)), dict(init=at(9)), dict(init=at(10), fin=at(10) + 64),
               dict(cu=at(11), fin=at(11)), dict(cu=at(9))):
        assert ssm(lib, **kw) == -4, kw
    for kw in (dict(pool=-1), dict(slots=None, pool=1), dict(pool=1 << 50), dict(n=1 << 30)):
        assert ssm_step(lib, **kw) == -2, kw
    assert ssm_step(lib, state=None) == -1 and ssm_step(lib, state=at(8) + 8) == -3 and ssm_step(lib, slots=at(10) + 2) == -3
    for kw in (dict(state=at(2)), dict(state=at(10)), dict(out=at(8))):
        assert ssm_step(lib, **kw) == -4, kw
    # The type of the states is part of the overlap rule.
    assert ssm(lib, init=at(10), fin=at(10) + 2 * 64 * 16 * 2, flags=258) == -4
    if no_gpu():
        assert ssm(lib, init=at(10), fin=at(10) + 2 * 64 * 16 * 2) == -5 and ssm(lib, init=at(10)) == -5
        assert ssm(lib, T=0, x=None, dt=None, B=None, C=None, D=None, z=None, out=None) == -5
        assert ssm_step(lib, pool=0, state=None) == -5


def test_scan_queries(lib):
    n = ctypes.c_int64(0)
    assert lib.kda_ssm_plan_segments(1, 16, 64, 1, 16, 0, None) == -1
    assert lib.kda_ssm_plan_segments(1, 16, 64, 3, 16, 0, ctypes.byref(n)) == -2
    assert lib.kda_ssm_workspace_bytes(1, 16, 64, 1, 16, 0, None) == -1
    assert lib.kda_ssm_workspace_bytes(1, -1, 64, 1, 16, 0, ctypes.byref(n)) == -2

    def need(N, T, dim, S, packed):
        assert lib.kda_ssm_workspace_bytes(N, T, dim, 1, S, packed, ctypes.byref(n)) == 0
        return n.value
    assert need(1, 16, 64, 16, 0) == 0 and need(1, 400, 12288, 16, 0) == 0
    assert need(2000, 16, 64, 16, 1) == 256            # many offsets: a verdict
    # Spans one after the other: a state each, sixteen at most for each sequence, and flags.
    assert need(1, 8192, 12288, 16, 0) <= 16 * 12288 * 16 * 4 + 16 * 384 * 4 + 12288 * 16 * 4 + 512
    # A cut never takes more than eight waves of CTAs, each with 32 channels' states.
    for dim, S in ((64, 16), (768, 16), (5120, 16), (768, 64)):
        states = 8 * 3 * 152 * 32 * (64 if S == 64 else 16) * 4
        assert 0 < need(1, 1 << 20, dim, S, 0) <= 1.1 * states + dim * S * 4 + 65536, (dim, S)


def test_python_refuses_host_tensors_and_shapes():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    f = lambda *s: t(*s, dt=torch.float32)  # noqa: E731
    with pytest.raises(ValueError, match="x must be a"):
        ops.conv_prefill(t(1, 4, 8), t(8, 4))
    with pytest.raises(ValueError, match="2 to 4"):
        ops.conv_prefill(t(1, 4, 8), t(8, 5))
    with pytest.raises(ValueError, match=r"B, T, D"):
        ops.conv_prefill(t(4, 8), t(8, 4))
    with pytest.raises(ValueError, match="activation"):
        ops.conv_prefill(t(1, 4, 8), t(8, 4), activation="sigmoid")
    with pytest.raises(ValueError, match="x must be a"):
        ops.conv_decode(t(4, 8), t(8, 4), t(5, 3, 8))
    with pytest.raises(ValueError, match=r"N, D"):
        ops.conv_decode(t(1, 4, 8), t(8, 4), t(5, 3, 8))
    args = (f(8, 16), t(1, 4, 1, 16), t(1, 4, 1, 16))
    with pytest.raises(ValueError, match="x must be a"):
        ops.ssm_prefill(t(1, 4, 8), t(1, 4, 8), *args)
    with pytest.raises(ValueError, match="groups"):
        ops.ssm_prefill(t(1, 4, 8), t(1, 4, 8), f(8, 16), t(1, 4, 3, 16), t(1, 4, 3, 16))
    with pytest.raises(ValueError, match="1 to 64"):
        ops.ssm_prefill(t(1, 4, 8), t(1, 4, 8), f(8, 65), t(1, 4, 1, 65), t(1, 4, 1, 65))
    with pytest.raises(ValueError, match=r"G, S"):
        ops.ssm_prefill(t(1, 4, 8), t(1, 4, 8), f(8, 16), t(1, 4, 16), t(1, 4, 16))
    with pytest.raises(ValueError, match="x must be a"):
        ops.ssm_decode(t(4, 8), t(4, 8), f(8, 16), t(4, 1, 16), t(4, 1, 16), f(5, 8, 16))
