"""Refusals of the operators around the prefill (no GPU needed): bad arguments
are turned away on the host, before any CUDA call.  Addresses passed here are
never dereferenced."""

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


def la(lib, q=at(0), k=at(1), v=at(2), g=at(3), init=None, out=at(4), fin=None, B=1, T=16, H=4, Hk=2, cu=None,
       flags=0):
    return lib.kda_la_prefill(q, k, v, g, init, out, fin, B, T, H, Hk, cu, 0.1, flags, None)


def test_la_prefill(lib):
    assert la(lib, flags=1) == -7 and la(lib, flags=8) == -7
    for kw in (dict(B=0), dict(T=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(H=1 << 50), dict(B=1 << 40, T=1 << 40),
               dict(T=1 << 31), dict(B=1 << 31)):
        assert la(lib, **kw) == -2, kw
    for name in ("q", "k", "v", "g", "out"):
        assert la(lib, **{name: None}) == -1, name
    for kw in (dict(q=at(0) + 8), dict(k=at(1) + 2), dict(v=at(2) + 4), dict(g=at(3) + 2), dict(out=at(4) + 8),
               dict(init=at(5) + 8), dict(fin=at(5) + 8), dict(cu=at(6) + 4)):
        assert la(lib, **kw) == -3, kw
    for kw in (dict(out=at(0) + 64), dict(out=at(2)), dict(fin=at(1)), dict(fin=at(4)),
               dict(init=at(5), fin=at(5) + 1024), dict(out=at(5), init=at(5)), dict(fin=at(6), cu=at(6))):
        assert la(lib, **kw) == -4, kw
    if no_gpu():
        assert la(lib) == -5
        assert la(lib, init=at(5), fin=at(5), flags=6) == -5
        assert la(lib, q=None, k=None, v=None, g=None, out=None, T=0) == -5
    # The type of the states is part of the overlap rule.
    assert la(lib, init=at(5), fin=at(5) + 4 * 128 * 128 * 2, flags=2) == -4


def test_la_queries(lib):
    n = ctypes.c_int64(0)
    assert lib.kda_la_plan_segments(1, 16, 0, 0, ctypes.byref(n)) == -2
    assert lib.kda_la_plan_segments(1, 16, 1, 0, None) == -1
    assert lib.kda_la_workspace_bytes(1, -1, 1, 0, ctypes.byref(n)) == -2
    assert lib.kda_la_workspace_bytes(1, 16, 1, 0, None) == -1
    assert lib.kda_la_workspace_bytes(1, 16, 1, 0, ctypes.byref(n)) == 0 and n.value == 0


def la_step(lib, q=at(0), k=at(1), v=at(2), g=at(3), state=at(4), slots=at(5), out=at(6), N=2, H=4, Hk=2, pool=3,
            flags=0):
    return lib.kda_la_decode(q, k, v, g, state, slots, out, N, H, Hk, pool, 0.1, flags, None)


def kda_step(lib, q=at(0), k=at(1), v=at(2), g=at(3), beta=at(7), state=at(4), slots=at(5), out=at(6), N=2, H=4,
             pool=3, flags=0):
    return lib.kda_decode(q, k, v, g, beta, state, slots, out, N, H, pool, flags, None)


@pytest.mark.parametrize("step", [la_step, kda_step])
def test_steps(lib, step):
    assert step(lib, flags=8) == -7
    for kw in (dict(N=-1), dict(H=0), dict(pool=-1), dict(slots=None, pool=1), dict(N=1 << 40), dict(pool=1 << 50),
               dict(H=1 << 50)):
        assert step(lib, **kw) == -2, kw
    for name in ("q", "k", "v", "g", "out", "state"):
        assert step(lib, **{name: None}) == -1, name
    for kw in (dict(q=at(0) + 8), dict(k=at(1) + 2), dict(v=at(2) + 4), dict(g=at(3) + 2), dict(out=at(6) + 8),
               dict(state=at(4) + 8), dict(slots=at(5) + 2)):
        assert step(lib, **kw) == -3, kw
    for kw in (dict(out=at(0)), dict(out=at(4) + 16), dict(state=at(1)), dict(state=at(5)), dict(out=at(3))):
        assert step(lib, **kw) == -4, kw
    if no_gpu():
        assert step(lib) == -5 and step(lib, flags=2) == -5 and step(lib, slots=None) == -5


def test_step_own_arguments(lib):
    assert la_step(lib, Hk=3) == -2 and la_step(lib, Hk=0) == -2
    assert la_step(lib, flags=1) == -7 and kda_step(lib, flags=4) == -7
    assert kda_step(lib, beta=None) == -1 and kda_step(lib, beta=at(7) + 1) == -3
    assert kda_step(lib, g=at(3) + 8) == -3 and kda_step(lib, out=at(7)) == -4


def gn(lib, x=at(0), w=at(1), z=at(2), out=at(3), rows=5, act=1, eps=1e-6, flags=0):
    return lib.kda_gated_norm(x, w, z, out, rows, act, eps, flags, None)


def test_gated_norm(lib):
    for kw in (dict(flags=1), dict(flags=32), dict(act=3), dict(act=-1), dict(eps=-1.0), dict(eps=float("nan"))):
        assert gn(lib, **kw) == -7, kw
    assert gn(lib, rows=-1) == -2 and gn(lib, rows=1 << 40) == -2
    for name in ("x", "w", "z", "out"):
        assert gn(lib, **{name: None}) == -1, name
    for kw in (dict(x=at(0) + 8), dict(w=at(1) + 8), dict(z=at(2) + 8), dict(out=at(3) + 8)):
        assert gn(lib, **kw) == -3, kw
    for kw in (dict(out=at(0) + 256), dict(out=at(2) + 256), dict(out=at(1))):
        assert gn(lib, **kw) == -4, kw
    if no_gpu():
        assert gn(lib) == -5 and gn(lib, out=at(0)) == -5 and gn(lib, out=at(2)) == -5
        assert gn(lib, z=None, act=0) == -5 and gn(lib, flags=24, act=2) == -5


def rn(lib, x=at(0), r=at(1), w=at(2), post=None, gate=None, out=at(3), ro=at(4), rows=5, dim=64, eps=1e-6, flags=0):
    return lib.kda_residual_norm(x, r, w, post, gate, out, ro, rows, dim, 1.0, eps, flags, None)


def test_residual_norm(lib):
    for kw in (dict(flags=1), dict(flags=16), dict(eps=-1.0), dict(eps=float("nan"))):
        assert rn(lib, **kw) == -7, kw
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=32769)):
        assert rn(lib, **kw) == -2, kw
    for name in ("x", "r", "w", "out", "ro"):
        assert rn(lib, **{name: None}) == -1, name
    for kw in (dict(x=at(0) + 8), dict(post=at(5) + 8), dict(gate=at(5) + 4), dict(ro=at(4) + 8)):
        assert rn(lib, **kw) == -3, kw
    for kw in (dict(out=at(0) + 128), dict(ro=at(1) + 128), dict(out=at(1)), dict(ro=at(0)), dict(ro=at(3)),
               dict(out=at(2)), dict(gate=at(5), ro=at(5)), dict(post=at(5), out=at(5))):
        assert rn(lib, **kw) == -4, kw
    if no_gpu():
        assert rn(lib) == -5 and rn(lib, out=at(0), ro=at(1)) == -5 and rn(lib, post=at(5), gate=at(6), flags=40) == -5


def test_python_refuses_host_tensors_and_shapes():
    t = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="q must be a contiguous"):
        ops.la_prefill(t(1, 4, 2, 128), t(1, 4, 2, 128), t(1, 4, 2, 128), t(1, 4, 2, dt=torch.float32))
    with pytest.raises(ValueError, match="heads"):
        ops.la_prefill(t(1, 4, 3, 128), t(1, 4, 3, 128), t(1, 4, 4, 128), t(4, dt=torch.float32))
    with pytest.raises(ValueError, match="128"):
        ops.la_prefill(t(1, 4, 2, 64), t(1, 4, 2, 64), t(1, 4, 2, 64), t(2, dt=torch.float32))
    with pytest.raises(ValueError, match="q must be a contiguous"):
        ops.la_decode(t(1, 2, 128), t(1, 2, 128), t(1, 2, 128), t(1, 2, dt=torch.float32), t(1, 2, 128, 128))
    with pytest.raises(ValueError, match="128"):
        ops.kda_decode(t(1, 128), t(1, 128), t(1, 128), t(1, 128), t(1), t(1, 2, 128, 128))
    with pytest.raises(ValueError, match="activation"):
        ops.gated_norm(t(2, 128), t(128), t(2, 128), activation="tanh")
    with pytest.raises(ValueError, match="128"):
        ops.gated_norm(t(2, 64), t(64), t(2, 64))
    with pytest.raises(ValueError, match="x must be a contiguous"):
        ops.residual_norm(t(2, 64), t(2, 64), t(64))


def test_packed_workspace_stays_small(lib):
    """Room for a cut only where one can be worth it, and for few states."""
    def need(N, T, H):
        n = ctypes.c_int64()
        assert lib.kda_la_workspace_bytes(N, T, H, 1, ctypes.byref(n)) == 0
        return n.value
    state = 128 * 128 * 4
    assert need(4, 2000, 8) == 256                        # nothing to decide
    assert need(8, 1 << 20, 128) <= 1024                  # a cut never pays: the order alone
    for H in (1, 6, 12, 32, 64):
        for T in (4096, 33333, 1 << 17, 1 << 20):
            segments = max(16 * 152 / H, T / (64 * 128)) + 8
            assert need(8, T, H) <= segments * H * state * 1.01 + 65536, (H, T)
