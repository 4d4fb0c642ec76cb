"""The wait of the linear-attention kernels is bounded in time: run out in the
test library, whose bound is 10^5 cycles, it must report and return within that
time.  The bound is a number of tries, each as long as the hardware suspends a
warp, so this is also what shows that the library's own two seconds are two."""

import ctypes

import pytest
import torch

from kimi_delta_attention_kda_gb300 import build

pytestmark = pytest.mark.gpu

KDA_DEV_PIPE_TIMEOUT = 2


def test_a_wait_runs_out_in_time():
    build.build()
    hooks = ctypes.CDLL(build.build_test_hooks())
    P = ctypes.c_void_p
    hooks.kda_test_wait_phase.argtypes = [P, P, P]
    hooks.kda_test_wait_phase.restype = ctypes.c_int
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    rc = hooks.kda_test_wait_phase(status.data_ptr(), out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    ended, ran_out, cycles = out.tolist()
    assert ended == 1                       # the completed barrier's wait
    assert ran_out == 1                     # the other one's
    # (Whole tries: down to half of the bound.)
    assert build.TEST_WAIT_BOUND_CYCLES / 2 <= cycles <= build.TEST_WAIT_BOUND_CYCLES
    assert int(status.item()) == KDA_DEV_PIPE_TIMEOUT
