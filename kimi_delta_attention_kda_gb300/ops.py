"""The operators around the prefill: per-head-decay linear attention, the
single-token steps, and the norms around a block.

Argument checks and marshalling only: the work runs in ``libkda.so``
(``include/kda.h``, "Operators around the prefill").  Every call is
asynchronous on ``stream`` (default: the current PyTorch stream), takes
contiguous CUDA tensors of the current device, and can be captured into a
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

_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream

# For a single token the checks and the marshalling cost more than the kernel:
# each operator first has one expression that is true of good arguments, and
# the checks that find the fault and name it run only where it is not.


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


def _device(name, t, dtype):
    """The device of the first argument, which has to be the current one."""
    _need(name, t, dtype, t.shape, t.get_device())
    if t.get_device() != _current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    return t.get_device()


def _stream(stream, dev):
    if stream is None:
        return _current_stream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _new(shape, dtype, dev, stream):
    """A new tensor in the memory of the stream that the call runs on: a block
    that another stream has just freed may still be in use there."""
    handle = _stream(stream, dev)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream(dev)):
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
    """
    qs, vs, gs, dev = q.shape, v.shape, g.shape, q.get_device()
    if not (dev >= 0 and len(qs) == 4 and qs[3] == HEAD_DIM and k.shape == qs and len(vs) == 4
            and vs[:2] == qs[:2] and vs[3] == HEAD_DIM and qs[2] > 0 and vs[2] % qs[2] == 0
            and (gs == vs[:3] or gs == vs[2:3])
            and q.dtype is _BF16 and k.dtype is _BF16 and v.dtype is _BF16 and g.dtype is _F32
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and g.is_contiguous()
            and k.get_device() == dev and v.get_device() == dev and g.get_device() == dev
            and (out is None or (out.dtype is _BF16 and out.shape == vs and out.is_contiguous()
                                 and out.get_device() == dev))
            and dev == _current_device()):
        if len(qs) != 4 or len(vs) != 4 or qs[3] != HEAD_DIM:
            raise ValueError("q and v must be [B, T, heads, 128]")
        if qs[2] < 1 or vs[2] % qs[2]:
            raise ValueError("the heads of v must be a multiple of the heads of q")
        dev = _device("q", q, _BF16)
        _need("k", k, _BF16, qs, dev)
        _need("v", v, _BF16, (qs[0], qs[1], vs[2], HEAD_DIM), dev)
        _need("g", g, _F32, vs[2:3] if len(gs) == 1 else vs[:3], dev)
        if out is not None:
            _need("out", out, _BF16, vs, dev)
    N, T, H, _ = vs
    flags = _lib.FLAG_G_PER_HEAD if len(gs) == 1 else 0
    if cu_seqlens is not None:
        if N != 1:
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
    elif output_final_state:
        shape = (N, H, HEAD_DIM, HEAD_DIM)
        final_state = (torch.empty(shape, dtype=state_dtype, device="cuda") if stream is None
                       else _new(shape, state_dtype, dev, stream))
    if out is None:
        out = torch.empty_like(v) if stream is None else _new(vs, _BF16, dev, stream)
    if state_dtype is _F32:
        flags |= _lib.FLAG_STATE_F32
    rc = _lib.load().kda_la_prefill(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), _ptr(init_state), out.data_ptr(),
        _ptr(final_state), N, T, H, qs[2], _ptr(cu_seqlens), _SCALE if scale is None else scale, flags,
        _current_stream(dev) if stream is None else _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_la_prefill")
    return out, final_state


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


def _good_step(q, k, v, g, state, slots, out, qs, vs, ss, dev):
    return (dev >= 0 and len(qs) == 3 and len(vs) == 3 and len(ss) == 4 and qs[2] == HEAD_DIM
            and vs[0] == qs[0] and vs[2] == HEAD_DIM and k.shape == qs
            and ss[1] == vs[1] and ss[2] == HEAD_DIM and ss[3] == HEAD_DIM
            and q.dtype is _BF16 and k.dtype is _BF16 and v.dtype is _BF16 and g.dtype is _F32
            and (state.dtype is _F32 or state.dtype is _BF16)
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and g.is_contiguous()
            and state.is_contiguous()
            and k.get_device() == dev and v.get_device() == dev and g.get_device() == dev
            and state.get_device() == dev
            and (qs[0] <= ss[0] if slots is None else
                 slots.dtype is torch.int32 and slots.shape == qs[:1] and slots.is_contiguous()
                 and slots.get_device() == dev)
            and (out is None or (out.dtype is _BF16 and out.shape == vs and out.is_contiguous()
                                 and out.get_device() == dev))
            and dev == _current_device())


def la_decode(q, k, v, g, state, slots=None, out=None, scale=None, stream=None):
    """One token per sequence of ``la_prefill``'s operation; returns ``out``
    and updates ``state`` in place.

    q, k: bf16 ``[N, Hk, 128]``; v: bf16 ``[N, H, 128]``; g: fp32 ``[N, H]`` or
    ``[H]``; state: fp32 or bf16 ``[pool, H, 128, 128]``; slots: int32 ``[N]`` on
    the device, the pool row of each sequence (no row twice; negative: a padding
    row, whose output is zero), or None for rows 0 .. N - 1.  A slot beyond the
    pool is treated as padding and sets ``KDA_DEV_BAD_SLOTS`` (``device_status``).
    """
    qs, vs, ss, gs, dev = q.shape, v.shape, state.shape, g.shape, q.get_device()
    if not (_good_step(q, k, v, g, state, slots, out, qs, vs, ss, dev) and qs[1] > 0 and vs[1] % qs[1] == 0
            and (gs == vs[:2] or gs == vs[1:2])):
        _check_step(q, k, v, g, state, slots, out, None, False)
    if out is None:
        out = torch.empty_like(v) if stream is None else _new(vs, _BF16, dev, stream)
    flags = ((_lib.FLAG_STATE_F32 if state.dtype is _F32 else 0) |
             (_lib.FLAG_G_PER_HEAD if len(gs) == 1 else 0))
    rc = _lib.load().kda_la_decode(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), state.data_ptr(),
        None if slots is None else slots.data_ptr(), out.data_ptr(), qs[0], vs[1], qs[1], ss[0],
        _SCALE if scale is None else scale, flags, _current_stream(dev) if stream is None else _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_la_decode")
    return out


def kda_decode(q, k, v, g, beta, state, slots=None, out=None, beta_is_logit=False, stream=None):
    """One token per sequence of ``kda_prefill``'s operation (q and k are
    L2-normalised inside); returns ``out`` and updates ``state`` in place.

    q, k, v: bf16 ``[N, H, 128]``; g: fp32 ``[N, H, 128]``; beta: bf16 ``[N, H]``;
    state and slots as for ``la_decode``: ``kda_prefill``'s final state (bf16) is
    such a state, and its fp32 copy keeps long generations from rounding it at
    every token.
    """
    qs, vs, ss, dev = q.shape, v.shape, state.shape, q.get_device()
    if not (_good_step(q, k, v, g, state, slots, out, qs, vs, ss, dev) and qs == vs and g.shape == vs
            and beta.dtype is _BF16 and beta.shape == vs[:2] and beta.is_contiguous() and beta.get_device() == dev):
        _check_step(q, k, v, g, state, slots, out, beta, True)
    if out is None:
        out = torch.empty_like(v) if stream is None else _new(vs, _BF16, dev, stream)
    flags = ((_lib.FLAG_STATE_F32 if state.dtype is _F32 else 0) |
             (_lib.FLAG_BETA_LOGIT if beta_is_logit else 0))
    rc = _lib.load().kda_decode(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(),
        None if slots is None else slots.data_ptr(), out.data_ptr(), qs[0], vs[1], ss[0], flags,
        _current_stream(dev) if stream is None else _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_decode")
    return out


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
    shape, dev, wt = x.shape, x.get_device(), weight.dtype
    if not (dev >= 0 and shape[-1:] == (HEAD_DIM,) and x.dtype is _BF16 and x.is_contiguous()
            and (wt is _F32 or wt is _BF16) and weight.shape == (HEAD_DIM,) and weight.is_contiguous()
            and weight.get_device() == dev
            and (not act or (gate.dtype is _BF16 and gate.shape == shape and gate.is_contiguous()
                             and gate.get_device() == dev))
            and (out is None or (out.dtype is _BF16 and out.shape == shape and out.is_contiguous()
                                 and out.get_device() == dev))
            and dev == _current_device()):
        if shape[-1:] != (HEAD_DIM,):
            raise ValueError("x must be [..., 128]")
        dev = _device("x", x, _BF16)
        _need("weight", weight, _FLOATS, (HEAD_DIM,), dev)
        if act:
            _need("gate", gate, _BF16, shape, dev)
        if out is not None:
            _need("out", out, _BF16, shape, dev)
    if out is None:
        out = torch.empty_like(x) if stream is None else _new(shape, _BF16, dev, stream)
    flags = (_lib.FLAG_WEIGHT_F32 if wt is _F32 else 0) | (_lib.FLAG_GATE_FIRST if gate_first else 0)
    rc = _lib.load().kda_gated_norm(
        x.data_ptr(), weight.data_ptr(), gate.data_ptr() if act else None, out.data_ptr(),
        x.numel() // HEAD_DIM, act, eps, flags, _current_stream(dev) if stream is None else _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_gated_norm")
    return out


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
    shape, dev, rt, wt = x.shape, x.get_device(), residual.dtype, weight.dtype
    ws = shape[-1:]
    if not (dev >= 0 and len(ws) == 1 and ws[0] > 0 and x.dtype is _BF16 and x.is_contiguous()
            and (rt is _F32 or rt is _BF16) and residual.shape == shape and residual.is_contiguous()
            and residual.get_device() == dev
            and (wt is _F32 or wt is _BF16) and weight.shape == ws and weight.is_contiguous()
            and weight.get_device() == dev
            and (post_weight is None or (post_weight.dtype is wt and post_weight.shape == ws
                                         and post_weight.is_contiguous() and post_weight.get_device() == dev))
            and (gate is None or (gate.dtype is wt and gate.shape == ws and gate.is_contiguous()
                                  and gate.get_device() == dev))
            and (out is None or (out.dtype is _BF16 and out.shape == shape and out.is_contiguous()
                                 and out.get_device() == dev))
            and (residual_out is None or (residual_out.dtype is rt and residual_out.shape == shape
                                          and residual_out.is_contiguous() and residual_out.get_device() == dev))
            and dev == _current_device()):
        if len(ws) != 1 or ws[0] < 1:
            raise ValueError("x must be [..., D]")
        dev = _device("x", x, _BF16)
        _need("residual", residual, _FLOATS, shape, dev)
        _need("weight", weight, _FLOATS, ws, dev)
        if post_weight is not None:
            _need("post_weight", post_weight, wt, ws, dev)
        if gate is not None:
            _need("gate", gate, wt, ws, dev)
        if out is not None:
            _need("out", out, _BF16, shape, dev)
        if residual_out is not None:
            _need("residual_out", residual_out, rt, shape, dev)
    if out is None:
        out = torch.empty_like(x) if stream is None else _new(shape, _BF16, dev, stream)
    if residual_out is None:
        residual_out = torch.empty_like(residual) if stream is None else _new(shape, rt, dev, stream)
    flags = (_lib.FLAG_WEIGHT_F32 if wt is _F32 else 0) | (_lib.FLAG_RESIDUAL_F32 if rt is _F32 else 0)
    D = ws[0]
    rc = _lib.load().kda_residual_norm(
        x.data_ptr(), residual.data_ptr(), weight.data_ptr(),
        None if post_weight is None else post_weight.data_ptr(), None if gate is None else gate.data_ptr(),
        out.data_ptr(), residual_out.data_ptr(), x.numel() // D, D, scale, eps, flags,
        _current_stream(dev) if stream is None else _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_residual_norm")
    return out, residual_out
