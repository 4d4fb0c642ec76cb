"""The scratch that a cut kda_la_prefill call may take (no GPU needed; planned as
on 152 SMs): one FP32 state an SM, the copies of initial states that a call in
place overwrites, and tables."""

import ctypes

import pytest
import torch

from kimi_delta_attention_kda_gb300 import _lib, build

SMS, STATE = 152, 128 * 128 * 4


@pytest.fixture(scope="module")
def need():
    build.build()
    lib = _lib.load()
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != SMS:
        pytest.skip("planned on a GPU with another number of SMs")

    def bytes_of(N, T, H, packed):
        n = ctypes.c_int64()
        assert lib.kda_la_workspace_bytes(N, T, H, int(packed), ctypes.byref(n)) == 0
        return n.value
    return bytes_of


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("N", [1, 8, 40])
@pytest.mark.parametrize("H", [1, 6, 32, 96])
def test_one_state_an_sm(need, N, H, packed):
    for T in (1, 4096, 33333, 1 << 20):
        # A head's decay over each span, and of a packed batch 16 bytes for each
        # part (N + spans), 4 for each span, 12 for each sequence, 256 for its
        # verdict: all rounded up to 256 bytes.
        tables = 4 * SMS + (16 * (N + SMS) + 4 * (SMS + 1) + 12 * N if packed else 0) + 6 * 256
        assert need(N, T, H, packed) <= (SMS + N * H) * STATE + tables, T


def test_a_cut_takes_its_states(need):
    """The bound above is not loose: T = 8192, 6 heads in 22 spans of 3 chunks each."""
    assert need(1, 8192, 6, False) == 22 * 6 * STATE + 3 * 256 + 6 * STATE


@pytest.mark.parametrize("T,H,cut", [(77, 6, False), (512, 2, False), (1024, 2, True), (1024, 12, True), (2048, 48, True),
                                     (8192, 6, True), (8192, 48, True), (8192, 76, False), (8192, 96, False),
                                     (16384, 64, True)])
def test_cut_where_it_was_measured_to_pay(need, T, H, cut):
    """Fixed layout, one sequence: on either side of the planner's costs."""
    assert (need(1, T, H, False) > 0) == cut
