"""The operators and Python's threads: the interpreter's lock is free while the
library is called, and calls from several threads, each on a stream of its own,
give the bits of calls from one."""

import ctypes
import importlib.util
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

HOLD = 0.4   # seconds of a stand-in for a native call that waits


@pytest.fixture(scope="module")
def kda():
    import kimi_delta_attention_kda_gb300 as m
    from kimi_delta_attention_kda_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.device_status()
    return m


@pytest.fixture(scope="module")
def slow(kda, tmp_path_factory):
    """The module of the calls on tensors once more, on entry points that only
    wait for HOLD seconds on the host."""
    from kimi_delta_attention_kda_gb300 import _lib
    _lib.load_torch_module()
    here = tmp_path_factory.mktemp("slow")
    src, lib, module = here / "hold.c", here / "hold.so", here / "_kda_torch.so"
    src.write_text("#include <time.h>\nint hold(void) { struct timespec t = {0, %d}; return nanosleep(&t, 0); }\n"
                   % int(HOLD * 1e9))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    shutil.copy(_lib.TORCH_PATH, module)
    spec = importlib.util.spec_from_file_location("_kda_torch", str(module))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    hold = ctypes.CDLL(str(lib))
    m.bind(*[ctypes.cast(hold.hold, ctypes.c_void_p).value] * 5)
    m.keep = hold
    return m


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16, device="cuda")


def f32(*s):
    return torch.zeros(s, device="cuda")


CALLS = {
    "la_prefill": lambda m: m.la_prefill(bf(1, 9, 2, 128), bf(1, 9, 2, 128), bf(1, 9, 2, 128), f32(1, 9, 2), None, None,
                                         None, None, True, True, 1.0, None),
    "la_decode": lambda m: m.la_decode(bf(2, 2, 128), bf(2, 2, 128), bf(2, 2, 128), f32(2, 2), f32(2, 2, 128, 128), None,
                                       None, 1.0, None),
    "kda_decode": lambda m: m.kda_decode(bf(2, 2, 128), bf(2, 2, 128), bf(2, 2, 128), f32(2, 2, 128), bf(2, 2),
                                         f32(2, 2, 128, 128), None, None, False, None),
    "gated_norm": lambda m: m.gated_norm(bf(3, 128), bf(128), None, 0, False, 1e-6, None, None),
    "residual_norm": lambda m: m.residual_norm(bf(3, 64), f32(3, 64), bf(64), None, None, 1.0, 1e-6, None, None, None),
}


@pytest.mark.parametrize("op", sorted(CALLS))
def test_other_threads_run_during_a_call(slow, op):
    ticks, done = [], threading.Event()

    def tick():
        while not done.is_set():
            ticks.append(time.monotonic())
            time.sleep(0.002)

    thread = threading.Thread(target=tick)
    thread.start()
    try:
        start = time.monotonic()
        result = CALLS[op](slow)
        end = time.monotonic()
    finally:
        done.set()
        thread.join()
    assert result is not None and not isinstance(result, int)
    assert end - start >= HOLD
    # A tenth of what an idle machine would do; none with the lock held.
    inside = [t for t in ticks if end - HOLD < t < end]
    assert len(inside) >= HOLD / 0.002 / 10


def test_calls_from_several_threads(kda):
    def work(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        q, k, v = (rnd(1, 300, 4, 128).bfloat16() for _ in range(3))
        g = -0.1 * torch.rand((1, 300, 4), generator=gen, device="cuda")
        tok = [rnd(6, 4, 128).bfloat16() for _ in range(3)]
        state, weight = rnd(6, 4, 128, 128), rnd(128).bfloat16()
        results = []
        for i in range(20):
            o, s = kda.la_prefill(q, k, v, g, init_state=state[:1])
            y = kda.la_decode(*tok, g[0, :6].contiguous(), state)
            z = kda.gated_norm(y, weight, tok[0])
            x, r = kda.residual_norm(z, y.float(), weight)
            results.append([o, s, y, z, x, r])
        torch.cuda.current_stream().synchronize()
        return results + [[state]]

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
        assert have is not None
        for xs, ys in zip(want, have):
            assert all(torch.equal(x, y) for x, y in zip(xs, ys))
