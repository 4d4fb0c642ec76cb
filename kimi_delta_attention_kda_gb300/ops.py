"""The operators around the prefill: per-head-decay linear attention, the
selective state space scan, the short causal convolution, the single-token
steps, and the norms around a block.

The work runs in ``libkda.so`` (``include/kda.h``, "Operators around the
prefill"); the arguments are checked and marshalled by ``csrc/kda_torch.cpp``,
which returns None where one is not what it should be: the checks here then
find the fault and name it.  Every call is
asynchronous on ``stream`` (default: the current PyTorch stream), takes
contiguous CUDA tensors of the current device (the convolution's and the scan's
inputs for each token may be parts of wider rows), and can be captured into a
CUDA graph.
"""

from __future__ import annotations

import torch

from . import _lib
from ._lib import KdaError

HEAD_DIM = 128
_SCALE = HEAD_DIM ** -0.5
_ACTIVATIONS = {"none": 0, "sigmoid": 1, "silu": 2}
_BF16, _F32 = torch.bfloat16, torch.float32
_FLOATS = (_F32, _BF16)


class _Native:
    """The functions of ``csrc/kda_torch.cpp``, loaded at the first use."""

    def __getattr__(self, name):
        module = _lib.load_torch_module()
        for op in ("la_prefill", "la_decode", "kda_decode", "gated_norm", "residual_norm", "conv_prefill",
                   "conv_decode", "ssm_prefill", "ssm_decode"):
            setattr(self, op, getattr(module, op))
        return getattr(module, name)


_native = _Native()


def _need(name, t, dtype, shape, dev):
    """Refuses anything but a contiguous CUDA tensor of this type (or one of
    these), shape and device."""
    types = dtype if type(dtype) is tuple else (dtype,)
    if not t.is_cuda or t.dtype not in types or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA tensor" % (name, " or ".join(str(d) for d in types)))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, list(shape), list(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on the device of the first argument" % name)


def _need_rows(name, t, dtype, shape, inner, dev):
    """Refuses anything but a CUDA tensor of this type, shape and device whose
    last ``inner`` sizes are a contiguous row, at one distance from token to token."""
    types = dtype if type(dtype) is tuple else (dtype,)
    if not t.is_cuda or t.dtype not in types:
        raise ValueError("%s must be a %s CUDA tensor" % (name, " or ".join(str(d) for d in types)))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, list(shape), list(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on the device of the first argument" % name)
    if not t.numel():
        return
    width, rows, step, fine = 1, 1, 0, True
    for i in range(t.dim() - 1, -1, -1):
        if t.shape[i] == 1:
            continue
        if i >= t.dim() - inner:
            fine = fine and t.stride(i) == width
            width *= t.shape[i]
        elif rows == 1:
            step, rows = t.stride(i), t.shape[i]
        else:
            fine = fine and t.stride(i) == rows * step
            rows *= t.shape[i]
    if not fine or (rows > 1 and step < width):
        raise ValueError("%s must have contiguous rows at one distance from token to token" % name)


def _device(name, t, dtype):
    """The device of the first argument, which has to be the current one."""
    _need(name, t, dtype, t.shape, t.get_device())
    if t.get_device() != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    return t.get_device()


def _handle(stream):
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _fail(rc, name):
    if type(rc) is int:
        raise KdaError(rc, "kda_" + name)
    raise ValueError("bad arguments for %s" % name)


def _new(shape, dtype, handle):
    """A new tensor in the memory of the stream that the call runs on: a block
    that another stream has just freed may still be in use there."""
    side = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(side):
        return torch.empty(shape, dtype=dtype, device="cuda")


def la_prefill(q, k, v, g, init_state=None, cu_seqlens=None, out=None, final_state=None,
               output_final_state=True, state_dtype=torch.float32, scale=None, stream=None):
    """Linear attention with one decay per head and token over whole prompts;
    returns ``(out, final_state)``:

        S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = scale * S_t q_t

    q, k: bf16 ``[B, T, Hk, 128]`` (Hk divides H; head h uses key head
    ``h // (H // Hk)``); v: bf16 ``[B, T, H, 128]``; g: fp32 ``[B, T, H]``
    log-decays <= 0, or ``[H]``, constant for each head; init_state:
    ``[N, H, 128, 128]`` (value rows x key columns), fp32 or bf16, or None for
    zeros; cu_seqlens: int64 ``[N + 1]`` on the device for the packed layout
    (then ``B == 1``).  ``final_state`` may be ``init_state``; a new one takes
    the type of ``init_state``, or ``state_dtype`` without one.  ``scale``
    defaults to 1/sqrt(128).

    The state is held in FP32; ``out`` takes one rounding to BF16 of the decayed
    scores and one of the state before each 128 tokens besides its own (2.4e-3 of
    its norm in all), and may be infinite where ``out / scale`` is above 2^79.
    """
    if stream is not None:
        _check_prefill(q, k, v, g, init_state, cu_seqlens, out, final_state, state_dtype)
        stream = _handle(stream)
        if out is None:
            out = _new(v.shape, _BF16, stream)
        if final_state is None and output_final_state:
            N = v.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            final_state = _new((N, v.shape[2], HEAD_DIM, HEAD_DIM),
                               state_dtype if init_state is None else init_state.dtype, stream)
    r = None
    if state_dtype is _F32 or state_dtype is _BF16:
        r = _native.la_prefill(q, k, v, g, init_state, cu_seqlens, out, final_state, output_final_state,
                               state_dtype is _F32, _SCALE if scale is None else scale, stream)
    if type(r) is not tuple:
        _check_prefill(q, k, v, g, init_state, cu_seqlens, out, final_state, state_dtype)
        _fail(r, "la_prefill")
    return r


def _check_prefill(q, k, v, g, init_state, cu_seqlens, out, final_state, state_dtype):
    """Names the fault in the arguments of la_prefill."""
    if q.dim() != 4 or v.dim() != 4 or q.shape[3] != HEAD_DIM:
        raise ValueError("q and v must be [B, T, heads, 128]")
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError("the heads of v must be a multiple of the heads of q")
    dev = _device("q", q, _BF16)
    _need("k", k, _BF16, q.shape, dev)
    _need("v", v, _BF16, (B, T, H, HEAD_DIM), dev)
    _need("g", g, _F32, (H,) if g.dim() == 1 else (B, T, H), dev)
    N = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed input needs B == 1")
        N = cu_seqlens.numel() - 1
        _need("cu_seqlens", cu_seqlens, torch.int64, (N + 1,), dev)
    if init_state is not None:
        _need("init_state", init_state, _FLOATS, (N, H, HEAD_DIM, HEAD_DIM), dev)
        state_dtype = init_state.dtype
    elif final_state is not None:
        state_dtype = final_state.dtype
    if state_dtype not in _FLOATS:
        raise ValueError("states are torch.float32 or torch.bfloat16")
    if final_state is not None:
        _need("final_state", final_state, state_dtype, (N, H, HEAD_DIM, HEAD_DIM), dev)
    if out is not None:
        _need("out", out, _BF16, v.shape, dev)


def _check_step(q, k, v, g, state, slots, out, beta, delta):
    """Names the fault in the arguments of a single-token step."""
    if q.dim() != 3 or v.dim() != 3 or q.shape[2] != HEAD_DIM or state.dim() != 4:
        raise ValueError("q and v must be [N, heads, 128], and state [pool, H, 128, 128]")
    dev = _device("q", q, _BF16)
    N, Hk, _ = q.shape
    H, pool = v.shape[1], state.shape[0]
    _need("q", q, _BF16, q.shape, dev)
    _need("k", k, _BF16, q.shape, dev)
    _need("v", v, _BF16, (N, H, HEAD_DIM), dev)
    _need("state", state, _FLOATS, (pool, H, HEAD_DIM, HEAD_DIM), dev)
    if slots is not None:
        _need("slots", slots, torch.int32, (N,), dev)
    elif N > pool:
        raise ValueError("state has fewer rows than there are sequences")
    if out is not None:
        _need("out", out, _BF16, (N, H, HEAD_DIM), dev)
    if delta:
        if Hk != H:
            raise ValueError("q must have the shape of v")
        _need("g", g, _F32, (N, H, HEAD_DIM), dev)
        _need("beta", beta, _BF16, (N, H), dev)
    else:
        if Hk < 1 or H % Hk:
            raise ValueError("the heads of v must be a multiple of the heads of q")
        _need("g", g, _F32, (H,) if g.dim() == 1 else (N, H), dev)


def la_decode(q, k, v, g, state, slots=None, out=None, scale=None, stream=None):
    """One token per sequence of ``la_prefill``'s operation; returns ``out``
    and updates ``state`` in place.

    q, k: bf16 ``[N, Hk, 128]``; v: bf16 ``[N, H, 128]``; g: fp32 ``[N, H]`` or
    ``[H]``; state: fp32 or bf16 ``[pool, H, 128, 128]``; slots: int32 ``[N]`` on
    the device, the pool row of each sequence (no row twice; negative: a padding
    row, whose output is zero), or None for rows 0 .. N - 1.  A slot beyond the
    pool is treated as padding and sets ``KDA_DEV_BAD_SLOTS`` (``device_status``).
    """
    if stream is not None:
        _check_step(q, k, v, g, state, slots, out, None, False)
        stream = _handle(stream)
        if out is None:
            out = _new(v.shape, _BF16, stream)
    r = _native.la_decode(q, k, v, g, state, slots, out, _SCALE if scale is None else scale, stream)
    if r is None or type(r) is int:
        _check_step(q, k, v, g, state, slots, out, None, False)
        _fail(r, "la_decode")
    return r


def kda_decode(q, k, v, g, beta, state, slots=None, out=None, beta_is_logit=False, stream=None):
    """One token per sequence of ``kda_prefill``'s operation (q and k are
    L2-normalised inside); returns ``out`` and updates ``state`` in place.

    q, k, v: bf16 ``[N, H, 128]``; g: fp32 ``[N, H, 128]``; beta: bf16 ``[N, H]``;
    state and slots as for ``la_decode``: ``kda_prefill``'s final state (bf16) is
    such a state, and its fp32 copy keeps long generations from rounding it at
    every token.
    """
    if stream is not None:
        _check_step(q, k, v, g, state, slots, out, beta, True)
        stream = _handle(stream)
        if out is None:
            out = _new(v.shape, _BF16, stream)
    r = _native.kda_decode(q, k, v, g, beta, state, slots, out, beta_is_logit, stream)
    if r is None or type(r) is int:
        _check_step(q, k, v, g, state, slots, out, beta, True)
        _fail(r, "decode")
    return r


def gated_norm(x, weight, gate=None, activation="sigmoid", gate_first=False, eps=1e-6, out=None,
               stream=None):
    """RMS norm over the last 128 channels with an output gate; returns ``out``:
    ``x / rms(x) * weight * act(gate)``, or with ``gate_first`` the norm of
    ``x * act(gate)`` times weight.

    x, gate, out: bf16 ``[..., 128]``; weight: bf16 or fp32 ``[128]``;
    activation: "sigmoid", "silu", or "none" (no gate).  Without a gate the
    activation is "none".  ``out`` may be ``x`` or ``gate``.
    """
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(sorted(_ACTIVATIONS)))
    act = _ACTIVATIONS[activation] if gate is not None else 0
    if stream is not None:
        _check_gated(x, weight, gate if act else None, out)
        stream = _handle(stream)
        if out is None:
            out = _new(x.shape, _BF16, stream)
    r = _native.gated_norm(x, weight, gate, act, gate_first, eps, out, stream)
    if r is None or type(r) is int:
        _check_gated(x, weight, gate if act else None, out)
        _fail(r, "gated_norm")
    return r


def _check_gated(x, weight, gate, out):
    """Names the fault in the arguments of gated_norm."""
    if x.dim() < 1 or x.shape[-1] != HEAD_DIM:
        raise ValueError("x must be [..., 128]")
    dev = _device("x", x, _BF16)
    _need("weight", weight, _FLOATS, (HEAD_DIM,), dev)
    if gate is not None:
        _need("gate", gate, _BF16, x.shape, dev)
    if out is not None:
        _need("out", out, _BF16, x.shape, dev)


def residual_norm(x, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-6, out=None,
                  residual_out=None, stream=None):
    """The residual sum between two blocks with the norms around it; returns
    ``(out, residual_out)``:

        u = x / rms(x) * post_weight          (x itself without post_weight)
        residual_out = residual + scale * gate * u
        out = residual_out / rms(residual_out) * weight

    x, out: bf16 ``[..., D]``, D up to 32768; residual: bf16 or fp32 of that
    shape; weight, post_weight, gate: bf16 or fp32 ``[D]``, all of one type.
    ``residual_out`` may be ``residual`` and ``out`` may be ``x``.
    """
    if stream is not None:
        _check_residual(x, residual, weight, post_weight, gate, out, residual_out)
        stream = _handle(stream)
        if out is None:
            out = _new(x.shape, _BF16, stream)
        if residual_out is None:
            residual_out = _new(x.shape, residual.dtype, stream)
    r = _native.residual_norm(x, residual, weight, post_weight, gate, scale, eps, out, residual_out, stream)
    if type(r) is not tuple:
        _check_residual(x, residual, weight, post_weight, gate, out, residual_out)
        _fail(r, "residual_norm")
    return r


def _check_residual(x, residual, weight, post_weight, gate, out, residual_out):
    """Names the fault in the arguments of residual_norm."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., D]")
    dev = _device("x", x, _BF16)
    wide = x.shape[-1:]
    _need("residual", residual, _FLOATS, x.shape, dev)
    _need("weight", weight, _FLOATS, wide, dev)
    for name, t in (("post_weight", post_weight), ("gate", gate)):
        if t is not None:
            _need(name, t, weight.dtype, wide, dev)
    if out is not None:
        _need("out", out, _BF16, x.shape, dev)
    if residual_out is not None:
        _need("residual_out", residual_out, residual.dtype, x.shape, dev)


def _silu(activation):
    if activation not in ("none", "silu"):
        raise ValueError("activation must be one of none, silu")
    return activation == "silu"


def conv_prefill(x, weight, bias=None, init_state=None, cu_seqlens=None, activation="silu", out=None,
                 final_state=None, output_final_state=True, stream=None):
    """The short causal convolution in front of a mixer, for each channel on its
    own; returns ``(out, final_state)``:

        out[t, d] = act(bias[d] + sum_j weight[d, j] x[t - W + 1 + j, d])

    x: bf16 ``[B, T, D]``, possibly a part of wider rows; weight: bf16 or fp32
    ``[D, W]``, W 2 to 4; bias: ``[D]`` of its type, or None; init_state: bf16
    ``[N, W - 1, D]``, the inputs before each sequence, oldest first, or None for
    zeros; cu_seqlens: int64 ``[N + 1]`` on the device for the packed layout
    (then ``B == 1``); activation: "silu" or "none".  ``final_state`` has each sequence's
    last W - 1 inputs and may be ``init_state``.
    """
    silu = _silu(activation)
    if stream is not None:
        _check_conv(x, weight, bias, init_state, cu_seqlens, out, final_state)
        stream = _handle(stream)
        if out is None:
            out = _new(x.shape, _BF16, stream)
        if final_state is None and output_final_state:
            N = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            final_state = _new((N, weight.shape[1] - 1, x.shape[2]), _BF16, stream)
    r = _native.conv_prefill(x, weight, bias, init_state, cu_seqlens, silu, out, final_state, output_final_state,
                             stream)
    if type(r) is not tuple:
        _check_conv(x, weight, bias, init_state, cu_seqlens, out, final_state)
        _fail(r, "conv_prefill")
    return r


def _check_filter(x, weight, bias, dims):
    """The device; names the fault in x and in the filter."""
    if x.dim() != dims or weight.dim() != 2 or not 2 <= weight.shape[1] <= 4:
        raise ValueError("x must be [%sD] and weight [D, 2 to 4]" % ("B, T, " if dims == 3 else "N, "))
    dev = x.get_device()
    _need_rows("x", x, _BF16, x.shape, 1, dev)
    if dev != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    _need("weight", weight, _FLOATS, (x.shape[-1], weight.shape[1]), dev)
    if bias is not None:
        _need("bias", bias, weight.dtype, x.shape[-1:], dev)
    return dev


def _count(x, cu_seqlens, dev):
    """The number of sequences of a prompt call."""
    if cu_seqlens is None:
        return x.shape[0]
    if x.shape[0] != 1:
        raise ValueError("packed input needs B == 1")
    _need("cu_seqlens", cu_seqlens, torch.int64, (cu_seqlens.numel(),), dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must have at least one offset")
    return cu_seqlens.numel() - 1


def _check_conv(x, weight, bias, init_state, cu_seqlens, out, final_state):
    """Names the fault in the arguments of conv_prefill."""
    dev = _check_filter(x, weight, bias, 3)
    state = (_count(x, cu_seqlens, dev), weight.shape[1] - 1, x.shape[2])
    for name, t, shape in (("init_state", init_state, state), ("out", out, x.shape), ("final_state", final_state, state)):
        if t is not None:
            _need(name, t, _BF16, shape, dev)


def conv_decode(x, weight, state, bias=None, slots=None, activation="silu", out=None, stream=None):
    """One token per sequence of ``conv_prefill``'s operation; returns ``out``
    and updates ``state`` in place: its rows move up by one, x becomes the last.

    x: bf16 ``[N, D]``, possibly a part of wider rows; state: bf16
    ``[pool, W - 1, D]``; weight and bias as for ``conv_prefill``, slots as for
    ``la_decode``.
    """
    silu = _silu(activation)
    if stream is not None:
        _check_conv_step(x, weight, state, bias, slots, out)
        stream = _handle(stream)
        if out is None:
            out = _new(x.shape, _BF16, stream)
    r = _native.conv_decode(x, weight, state, bias, slots, silu, out, stream)
    if r is None or type(r) is int:
        _check_conv_step(x, weight, state, bias, slots, out)
        _fail(r, "conv_decode")
    return r


def _check_slots(N, state, slots, dev):
    if slots is not None:
        _need("slots", slots, torch.int32, (N,), dev)
    elif N > state.shape[0]:
        raise ValueError("state has fewer rows than there are sequences")


def _check_conv_step(x, weight, state, bias, slots, out):
    """Names the fault in the arguments of conv_decode."""
    dev = _check_filter(x, weight, bias, 2)
    if state.dim() != 3:
        raise ValueError("state must be [pool, W - 1, D]")
    _need("state", state, _BF16, (state.shape[0], weight.shape[1] - 1, x.shape[1]), dev)
    _check_slots(x.shape[0], state, slots, dev)
    if out is not None:
        _need("out", out, _BF16, x.shape, dev)


def ssm_prefill(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, init_state=None, cu_seqlens=None,
                out=None, final_state=None, output_final_state=True, state_dtype=torch.float32, stream=None):
    """The selective state space scan over whole prompts, a linear recurrence
    whose decay differs in every channel d and state n; returns ``(out,
    final_state)``:

        s = softplus(dt + dt_bias)             (without dt_softplus the sum itself)
        h[d, n] = exp(s[d] A[d, n]) h[d, n] + s[d] x[d] B[g, n]
        out[d] = (sum_n C[g, n] h[d, n] + D[d] x[d]) silu(z[d])

    x, z: bf16 ``[B, T, dim]`` (z may be None: no gate); dt: bf16 or fp32 of that
    shape; A: fp32 ``[dim, S]``, S up to 64; B, C: both bf16 or fp32 ``[B, T, G, S]``
    (G divides dim; channel d has group ``g = d // (dim // G)``); D, dt_bias: fp32
    ``[dim]`` or None; init_state: ``[N, dim, S]``, fp32 or bf16, or None for zeros;
    cu_seqlens: int64 ``[N + 1]`` on the device for the packed layout (then
    ``B == 1``).  x, dt, B, C and z may be parts of wider rows.  ``final_state`` may
    be ``init_state``; a new one takes its type, or ``state_dtype`` without one.

    States and sums are FP32.  A rate of minus infinity clears its state at every
    step above 1e-36; a step of 0 leaves all states as they are.
    """
    if stream is not None:
        _check_ssm(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens, out, final_state, state_dtype)
        stream = _handle(stream)
        if out is None:
            out = _new(x.shape, _BF16, stream)
        if final_state is None and output_final_state:
            N = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
            final_state = _new((N,) + A.shape, state_dtype if init_state is None else init_state.dtype, stream)
    r = None
    if state_dtype is _F32 or state_dtype is _BF16:
        r = _native.ssm_prefill(x, dt, A, B, C, D, z, dt_bias, dt_softplus, init_state, cu_seqlens, out, final_state,
                                output_final_state, state_dtype is _F32, stream)
    if type(r) is not tuple:
        _check_ssm(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens, out, final_state, state_dtype)
        _fail(r, "ssm_prefill")
    return r


def _check_scan(x, dt, A, B, C, D, z, dt_bias, dims):
    """The device; names the fault in what both forms of the scan read."""
    if x.dim() != dims or B.dim() != dims + 1 or A.dim() != 2:
        raise ValueError("x must be [%sdim], A [dim, S], and B [%sG, S]" % (("B, T, " if dims == 3 else "N, ",) * 2))
    dim, S, G = x.shape[-1], A.shape[1], B.shape[-2]
    if not 1 <= S <= 64:
        raise ValueError("A must be [dim, 1 to 64]")
    if G < 1 or dim % G:
        raise ValueError("the groups of B must divide the channels of x")
    dev = x.get_device()
    _need_rows("x", x, _BF16, x.shape, 1, dev)
    if dev != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    _need_rows("dt", dt, _FLOATS, x.shape, 1, dev)
    _need("A", A, _F32, (dim, S), dev)
    _need_rows("B", B, _FLOATS, x.shape[:-1] + (G, S), 2, dev)
    _need_rows("C", C, B.dtype, x.shape[:-1] + (G, S), 2, dev)
    if z is not None:
        _need_rows("z", z, _BF16, x.shape, 1, dev)
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            _need(name, t, _F32, (dim,), dev)
    return dev


def _check_ssm(x, dt, A, B, C, D, z, dt_bias, init_state, cu_seqlens, out, final_state, state_dtype):
    """Names the fault in the arguments of ssm_prefill."""
    dev = _check_scan(x, dt, A, B, C, D, z, dt_bias, 3)
    state = (_count(x, cu_seqlens, dev),) + A.shape
    if init_state is not None:
        _need("init_state", init_state, _FLOATS, state, dev)
        state_dtype = init_state.dtype
    elif final_state is not None:
        state_dtype = final_state.dtype
    if state_dtype not in _FLOATS:
        raise ValueError("states are torch.float32 or torch.bfloat16")
    if final_state is not None:
        _need("final_state", final_state, state_dtype, state, dev)
    if out is not None:
        _need("out", out, _BF16, x.shape, dev)


def ssm_decode(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=True, slots=None, out=None,
               stream=None):
    """One token per sequence of ``ssm_prefill``'s operation; returns ``out`` and
    updates ``state`` in place.

    x, dt, z: ``[N, dim]``; B, C: ``[N, G, S]``; state: fp32 or bf16
    ``[pool, dim, S]``; the rest as for ``ssm_prefill``, slots as for ``la_decode``.
    """
    if stream is not None:
        _check_ssm_step(x, dt, A, B, C, D, z, dt_bias, state, slots, out)
        stream = _handle(stream)
        if out is None:
            out = _new(x.shape, _BF16, stream)
    r = _native.ssm_decode(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, slots, out, stream)
    if r is None or type(r) is int:
        _check_ssm_step(x, dt, A, B, C, D, z, dt_bias, state, slots, out)
        _fail(r, "ssm_decode")
    return r


def _check_ssm_step(x, dt, A, B, C, D, z, dt_bias, state, slots, out):
    """Names the fault in the arguments of ssm_decode."""
    dev = _check_scan(x, dt, A, B, C, D, z, dt_bias, 2)
    if state.dim() != 3:
        raise ValueError("state must be [pool, dim, S]")
    _need("state", state, _FLOATS, (state.shape[0],) + A.shape, dev)
    _check_slots(x.shape[0], state, slots, dev)
    if out is not None:
        _need("out", out, _BF16, x.shape, dev)
