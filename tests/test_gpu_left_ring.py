"""A kernel that gives up on a ring of copies (the streaming residual norm, after
a wait that ran out) first waits, within the same bound, for the copies still
under way: none may write to shared memory that the CTA has left.  The norm's
own waits cannot be made to run out without a fault, so what it calls then is
run in the test library."""

import ctypes

import pytest
import torch

from kimi_delta_attention_kda_gb300 import build

pytestmark = pytest.mark.gpu

KDA_DEV_PIPE_TIMEOUT = 2


@pytest.mark.parametrize("filled,left", [(3, 3), (2, 2), (1, 1), (0, 0), (2, 3), (0, 1)])
def test_copies_under_way_are_waited_for(filled, left):
    build.build()
    hooks = ctypes.CDLL(build.build_test_hooks())
    P, I = ctypes.c_void_p, ctypes.c_int
    hooks.kda_test_left_ring.argtypes = [P, I, I, P, P, P]
    hooks.kda_test_left_ring.restype = I
    src = torch.randint(0, 256, (4096,), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    rc = hooks.kda_test_left_ring(src.data_ptr(), filled, left, status.data_ptr(), out.data_ptr(),
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()                # returns: no wait hung
    all_came, same = out.tolist()
    assert all_came == (filled >= left)     # a copy that was never started runs out
    assert int(status.item()) == (0 if all_came else KDA_DEV_PIPE_TIMEOUT)
    if all_came:
        assert same == 1
