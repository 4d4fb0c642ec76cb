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

# For a single token the checks and the marshalling cost more than the kernel:
# one expression a tensor, and its message is made only where it fails.


def _bad(t, dtype, shape, dev):
    """Whether `t` is anything but a contiguous CUDA tensor of this type (or one
    of these), shape and device."""
    return (t.get_device() != dev or (t.dtype is not dtype and t.dtype not in _types(dtype))
            or t.shape != shape or not t.is_contiguous())


def _types(dtype):
    return dtype if type(dtype) is tuple else (dtype,)


def _refuse(name, t, dtype, shape, dev):
    if not t.is_cuda or t.dtype not in _types(dtype) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA tensor"
                         % (name, " or ".join(str(d) for d in _types(dtype))))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, list(shape), list(t.shape)))
    raise ValueError("%s must be on the device of the first argument" % name)


def _need(name, t, dtype, shape, dev):
    if _bad(t, dtype, shape, dev):
        _refuse(name, t, dtype, shape, dev)


def _device(name, t, dtype):
    """The device of the first argument, which has to be the current one."""
    dev = t.get_device()
    if dev < 0:
        _refuse(name, t, dtype, t.shape, dev)
    if dev != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current CUDA device")
    return dev


def _stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _new(shape, dtype, dev, stream):
    """A new tensor in the memory of the stream that the call runs on: a block
    that another stream has just freed may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
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
    if q.dim() != 4 or v.dim() != 4 or q.shape[3] != HEAD_DIM:
        raise ValueError("q and v must be [B, T, heads, 128]")
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    if Hk < 1 or H % Hk:
        raise ValueError("the heads of v must be a multiple of the heads of q")
    dev = _device("q", q, _BF16)
    _need("q", q, _BF16, q.shape, dev)
    _need("k", k, _BF16, q.shape, dev)
    _need("v", v, _BF16, (B, T, H, HEAD_DIM), dev)
    flags = 0
    if g.dim() == 1:
        _need("g", g, _F32, (H,), dev)
        flags = _lib.FLAG_G_PER_HEAD
    else:
        _need("g", g, _F32, (B, T, H), dev)
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
    elif output_final_state:
        final_state = _new((N, H, HEAD_DIM, HEAD_DIM), state_dtype, dev, stream)
    if out is None:
        out = _new(v.shape, _BF16, dev, stream)
    else:
        _need("out", out, _BF16, v.shape, dev)
    if state_dtype is _F32:
        flags |= _lib.FLAG_STATE_F32
    rc = _lib.load().kda_la_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(init_state), _ptr(out),
                                    _ptr(final_state), N, T, H, Hk, _ptr(cu_seqlens),
                                    _SCALE if scale is None else scale, flags, _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_la_prefill")
    return out, final_state


def _step_args(q, k, v, state, slots, out, stream):
    """Checks of q, k, v, state and slots of a single-token step;
    (device, N, H, Hk, pool, out)."""
    if q.dim() != 3 or v.dim() != 3 or q.shape[2] != HEAD_DIM or state.dim() != 4:
        raise ValueError("q and v must be [N, heads, 128], and state [pool, H, 128, 128]")
    dev = _device("q", q, _BF16)
    shape = q.shape
    N, Hk, _ = shape
    H, pool = v.shape[1], state.shape[0]
    _need("q", q, _BF16, shape, dev)
    _need("k", k, _BF16, shape, dev)
    _need("v", v, _BF16, (N, H, HEAD_DIM), dev)
    _need("state", state, _FLOATS, (pool, H, HEAD_DIM, HEAD_DIM), dev)
    if slots is not None:
        _need("slots", slots, torch.int32, (N,), dev)
    elif N > pool:
        raise ValueError("state has fewer rows than there are sequences")
    if out is None:
        out = _new(v.shape, _BF16, dev, stream)
    else:
        _need("out", out, _BF16, (N, H, HEAD_DIM), dev)
    return dev, N, H, Hk, pool, out


def la_decode(q, k, v, g, state, slots=None, out=None, scale=None, stream=None):
    """One token per sequence of ``la_prefill``'s operation; returns ``out``
    and updates ``state`` in place.

    q, k: bf16 ``[N, Hk, 128]``; v: bf16 ``[N, H, 128]``; g: fp32 ``[N, H]`` or
    ``[H]``; state: fp32 or bf16 ``[pool, H, 128, 128]``; slots: int32 ``[N]`` on
    the device, the pool row of each sequence (no row twice; negative: a padding
    row, whose output is zero), or None for rows 0 .. N - 1.  A slot beyond the
    pool is treated as padding and sets ``KDA_DEV_BAD_SLOTS`` (``device_status``).
    """
    dev, N, H, Hk, pool, out = _step_args(q, k, v, state, slots, out, stream)
    if Hk < 1 or H % Hk:
        raise ValueError("the heads of v must be a multiple of the heads of q")
    flags = _lib.FLAG_STATE_F32 if state.dtype is torch.float32 else 0
    if g.dim() == 1:
        _need("g", g, _F32, (H,), dev)
        flags |= _lib.FLAG_G_PER_HEAD
    else:
        _need("g", g, _F32, (N, H), dev)
    rc = _lib.load().kda_la_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state), _ptr(slots),
                                   _ptr(out), N, H, Hk, pool, _SCALE if scale is None else scale,
                                   flags, _stream(stream, dev))
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
    dev, N, H, Hk, pool, out = _step_args(q, k, v, state, slots, out, stream)
    if Hk != H:
        raise ValueError("q must have the shape of v")
    _need("g", g, _F32, (N, H, HEAD_DIM), dev)
    _need("beta", beta, _BF16, (N, H), dev)
    flags = ((_lib.FLAG_STATE_F32 if state.dtype is torch.float32 else 0) |
             (_lib.FLAG_BETA_LOGIT if beta_is_logit else 0))
    rc = _lib.load().kda_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                _ptr(slots), _ptr(out), N, H, pool, flags, _stream(stream, dev))
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
    if x.dim() < 1 or x.shape[-1] != HEAD_DIM:
        raise ValueError("x must be [..., 128]")
    dev = _device("x", x, _BF16)
    shape = x.shape
    _need("x", x, _BF16, shape, dev)
    _need("weight", weight, _FLOATS, (HEAD_DIM,), dev)
    if act:
        _need("gate", gate, _BF16, shape, dev)
    if out is None:
        out = _new(shape, _BF16, dev, stream)
    else:
        _need("out", out, _BF16, shape, dev)
    flags = ((_lib.FLAG_WEIGHT_F32 if weight.dtype is torch.float32 else 0) |
             (_lib.FLAG_GATE_FIRST if gate_first else 0))
    rc = _lib.load().kda_gated_norm(_ptr(x), _ptr(weight), _ptr(gate) if act else None, _ptr(out),
                                    x.numel() // HEAD_DIM, act, eps, flags, _stream(stream, dev))
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
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., D]")
    dev = _device("x", x, _BF16)
    shape = x.shape
    D = shape[-1]
    _need("x", x, _BF16, shape, dev)
    _need("residual", residual, _FLOATS, shape, dev)
    _need("weight", weight, _FLOATS, (D,), dev)
    if post_weight is not None:
        _need("post_weight", post_weight, weight.dtype, (D,), dev)
    if gate is not None:
        _need("gate", gate, weight.dtype, (D,), dev)
    if out is None:
        out = _new(shape, _BF16, dev, stream)
    else:
        _need("out", out, _BF16, shape, dev)
    if residual_out is None:
        residual_out = _new(shape, residual.dtype, dev, stream)
    else:
        _need("residual_out", residual_out, residual.dtype, shape, dev)
    flags = ((_lib.FLAG_WEIGHT_F32 if weight.dtype is torch.float32 else 0) |
             (_lib.FLAG_RESIDUAL_F32 if residual.dtype is torch.float32 else 0))
    rc = _lib.load().kda_residual_norm(_ptr(x), _ptr(residual), _ptr(weight), _ptr(post_weight),
                                       _ptr(gate), _ptr(out), _ptr(residual_out), x.numel() // D, D,
                                       scale, eps, flags, _stream(stream, dev))
    if rc != 0:
        raise KdaError(rc, "kda_residual_norm")
    return out, residual_out
