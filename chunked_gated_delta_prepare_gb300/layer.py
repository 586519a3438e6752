"""libgdr's layer operators (include/gdr.h, "the layer around the recurrence") on torch tensors.

    norm_forward, norm_backward               root-mean-square norm, residual, 8-bit output
    conv_forward, conv_backward, conv_step    short causal convolution
    ssm_forward, ssm_backward, ssm_step       selective state space scan
    delta_step                                the gated delta rule for one token
    lru_forward, lru_backward, lru_step       gated linear recurrence
    layernorm_forward, layernorm_backward     layer norm, residual
    gated_norm_forward, gated_norm_backward   norm of a recurrence's output, times a gate

The arithmetic runs in libgdr's CUDA kernels; binding/layer_binding.cpp checks the arguments and calls them, and a
missing library raises.  Each call takes device tensors, allocates its outputs (and a workspace, unless one is given)
and returns as soon as its kernels are queued on the current stream of the tensors' device, or on `stream` (a stream of
that device, or its handle), to which the outputs and the workspace then belong.  Shapes, types and devices that do not
fit raise ValueError; what the library refuses raises GdrError.

Inputs of tokens may be slices of a wider projection ([T, D] or [B, T, D] views with contiguous columns and one
stride for all rows); views with other strides are copied first, and so are gradients that are not contiguous.
States are changed in place and must be contiguous.
"""
from __future__ import annotations

import functools
import importlib.machinery
import importlib.util
import os
import threading
from typing import NamedTuple

import torch

from .gdr import LIB_PATH, load

BINDING_PATH = os.path.join(os.path.dirname(LIB_PATH), "_gdr_layer.so")

_binding = None
_lock = threading.Lock()


def _native():
    """The built binding, loaded on first use.  Raises if it is missing."""
    global _binding
    if _binding is not None:
        return _binding
    with _lock:
        if _binding is None:
            load()
            if not os.path.exists(BINDING_PATH):
                raise RuntimeError(f"the layer binding is not built ({BINDING_PATH} missing); run __graft_entry__.build() "
                                   "or python -m chunked_gated_delta_prepare_gb300.build")
            loader = importlib.machinery.ExtensionFileLoader("_gdr_layer", BINDING_PATH)
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_gdr_layer", loader))
            loader.exec_module(module)
            _binding = module
    return _binding


def _streamed(f):
    """Adds `stream` to a call: allocations and kernels of the call then belong to that stream, one of the tensors' device."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        device = next((t.device for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)), None)
        if device is None or device.type != "cuda":
            return f(*args, **kw)                    # which refuses them
        if isinstance(stream, int):                  # a handle says nothing of its device, and the current one may be another
            stream = torch.cuda.ExternalStream(stream, device=device)
        elif stream.device != device:
            raise ValueError(f"stream: a stream of {device} is needed, got one of {stream.device}")
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


# ---------------------------------------------------------------- root-mean-square norm

@_streamed
def norm_forward(x, weight, residual=None, *, eps=1e-6, quant=None, want_y=True):
    """y, r, y8, scales = norm_forward(x, weight, residual): the norm of s = x + residual over the last dimension.

    y = s * weight / sqrt(mean(s^2) + eps) in x's type (None with want_y=False); r = s in x's type, the new residual
    (x itself without a residual).  quant: None, "row" or a group of 32, 64 or 128 columns; then y8 is y / scale in
    float8_e4m3fn and scales fp32 holds one scale a row [..., 1] or a group [..., ceil(D / group)].
    """
    if quant is None:
        group = -1
    elif quant == "row":
        group = 0
    elif isinstance(quant, int) and quant > 0:
        group = quant
    else:
        raise ValueError(f"quant: None, 'row' or a number of columns is needed, got {quant!r}")
    y, r, y8, scales = _native().norm_forward(x, weight, residual, eps, group, want_y)
    return y, x if r is None else r, y8, scales


@_streamed
def norm_backward(dy, r, weight, d_r=None, *, eps=1e-6, workspace=None):
    """dx, dweight = norm_backward(dy, r, weight, d_r): from the forward's r, the gradient dy of y and the gradient d_r
    that reaches r by other ways.  dx is the gradient of x and of the residual alike; dweight is fp32."""
    return _native().norm_backward(dy, r, weight, d_r, eps, workspace)


# ---------------------------------------------------------------- short causal convolution

@_streamed
def conv_forward(x, weight, bias=None, state=None, *, silu=True, cu_seqlens=None, want_state=True):
    """y, state_out = conv_forward(x, weight, bias, state): each channel's tokens with the W taps of its weight row.

    x [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); weight [D, W] (W = 2, 3 or 4) and bias
    [D] in x's type; state [n, W - 1, D]: the inputs before the first token, oldest first (None: zero).  state_out has
    the last W - 1 inputs of each sequence (None with want_state=False)."""
    return _native().conv_forward(x, weight, bias, state, silu, cu_seqlens, want_state)


@_streamed
def conv_backward(x, weight, bias, dy, state=None, d_state_out=None, *, silu=True, cu_seqlens=None, workspace=None):
    """dx, dweight, dbias, dstate = conv_backward(x, weight, bias, dy, state, d_state_out): the gradient of
    conv_forward's y and state_out (d_state_out None: unused).  dweight and dbias are fp32; dbias is None without a
    bias, dstate without a state."""
    return _native().conv_backward(x, weight, bias, dy, state, d_state_out, silu, cu_seqlens, workspace)


@_streamed
def conv_step(x, weight, bias, state, *, silu=True, slots=None):
    """y = conv_step(x, weight, bias, state): one token x [n, D] of n sequences.  state [pool, W - 1, D] is shifted in
    place, row i using state slots[i] (device int32; None: state i); a slot outside the pool marks a padding row."""
    return _native().conv_step(x, weight, bias, state, silu, slots)


# ---------------------------------------------------------------- selective state space scan

@_streamed
def ssm_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True, cu_seqlens=None,
                want_h_final=True, workspace=None):
    """y, h_final = ssm_forward(x, dt, A, B, C, D, z, dt_bias, h0): the selective state space scan.

    x, dt, z [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); B, C [..., G, N], the D / G channels
    of a group sharing one; A [D, N], D [D], dt_bias [D] fp32; h0 [n, D, N] fp32 (None: zero).
        Delta = softplus(dt + dt_bias);  h = exp(Delta A) h + Delta x B;  y = (C.h + D x) silu(z)
    y is in the io type, h_final [n, D, N] fp32 (None with want_h_final=False)."""
    return _native().ssm_forward(x, dt, A, B, C, D, z, dt_bias, h0, softplus, cu_seqlens, want_h_final, workspace)


class SsmGrads(NamedTuple):
    dx: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: torch.Tensor | None
    dz: torch.Tensor | None
    ddt_bias: torch.Tensor | None
    dh0: torch.Tensor | None


@_streamed
def ssm_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, h0=None, dh_final=None, *, softplus=True,
                 cu_seqlens=None, workspace=None) -> SsmGrads:
    """The gradient of ssm_forward's y and h_final (dh_final None: unused), from the forward's inputs alone.  dx, ddt, dB,
    dC, dz are in the io type, the others fp32; those of inputs that are None are None."""
    return SsmGrads(*_native().ssm_backward(x, dt, A, B, C, dy, D, z, dt_bias, h0, dh_final, softplus, cu_seqlens,
                                            workspace))


@_streamed
def ssm_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, softplus=True, slots=None):
    """y = ssm_step(x, dt, A, B, C, h, D, z, dt_bias): one token of n rows, x, dt, z [n, D], B, C [n, G, N].  h [pool, D,
    N] fp32 is changed in place, row i using state slots[i] (device int32; None: state i); a slot outside the pool marks
    a padding row, whose y is zero."""
    return _native().ssm_step(x, dt, A, B, C, h, D, z, dt_bias, softplus, slots)


# ---------------------------------------------------------------- the gated delta rule, one token

@_streamed
def delta_step(q, k, v, g, beta, h, *, scale=None, slots=None):
    """o = delta_step(q, k, v, g, beta, h): one token of B rows, as forward() computes it for T = 1.

    q, k [B, H, K], v [B, HV, V] (slices of a wider [B, ...] row are used in place), beta [B, HV] in the io type;
    g [B, HV] or [B, HV, K] fp32.  h [pool, HV, K, V] fp32 is changed in place, row i using state slots[i] (device
    int32; None: state i); a slot outside the pool marks a padding row, whose o is zero."""
    return _native().delta_step(q, k, v, g, beta, h, scale, slots)


# ---------------------------------------------------------------- gated linear recurrence

@_streamed
def lru_forward(x, r, i=None, lam=None, h0=None, *, c=8.0, cu_seqlens=None, want_h_final=True, want_kept=False,
                workspace=None):
    """y, h_final, kept = lru_forward(x, r, i, lam, h0): the gated linear recurrence, one state a channel.

    x, r, i [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); lam [D] fp32; h0 [n, D] fp32 (None:
    zero).  With g = sigmoid(i) (1 without i):
        with lam:     log a = -c softplus(lam) sigmoid(r);  h = a h + sqrt(1 - a^2) g x
        without lam:  a = sigmoid(r);                       h = a h + (1 - a) g x
    y is h in the io type, h_final [n, D] fp32 (None with want_h_final=False).  kept: with want_kept=True the states that
    lru_backward starts its tiles from, fp32, one row for 128 tokens."""
    return _native().lru_forward(x, r, i, lam, h0, c, cu_seqlens, want_h_final, want_kept, workspace)


class LruGrads(NamedTuple):
    dx: torch.Tensor
    dr: torch.Tensor
    di: torch.Tensor | None
    dlam: torch.Tensor | None
    dh0: torch.Tensor | None


@_streamed
def lru_backward(x, r, i, lam, dy, h0=None, dh_final=None, kept=None, *, c=8.0, cu_seqlens=None,
                 workspace=None) -> LruGrads:
    """The gradient of lru_forward's y and h_final (dh_final None: unused), from the forward's inputs and its kept states
    (None: they are formed again).  dx, dr, di are in the io type, dlam and dh0 fp32; those of inputs that are None are
    None."""
    return LruGrads(*_native().lru_backward(x, r, i, lam, dy, h0, dh_final, kept, c, cu_seqlens, workspace))


@_streamed
def lru_step(x, r, i, lam, h, *, c=8.0, slots=None):
    """y = lru_step(x, r, i, lam, h): one token of n rows, x, r, i [n, D].  h [pool, D] fp32 is changed in place, row k
    using state slots[k] (device int32; None: state k); a slot outside the pool marks a padding row, whose y is zero."""
    return _native().lru_step(x, r, i, lam, h, c, slots)


# ---------------------------------------------------------------- layer norm

@_streamed
def layernorm_forward(x, weight, bias=None, residual=None, *, eps=1e-5, want_y=True):
    """y, r = layernorm_forward(x, weight, bias, residual): the layer norm of s = x + residual over the last dimension.

    y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias in x's type (None with want_y=False); r = s in x's type, the
    new residual (x itself without a residual)."""
    y, r = _native().layernorm_forward(x, weight, bias, residual, eps, want_y)
    return y, x if r is None else r


@_streamed
def layernorm_backward(dy, r, weight, d_r=None, *, eps=1e-5, workspace=None):
    """dx, dweight, dbias = layernorm_backward(dy, r, weight, d_r): from the forward's r, the gradient dy of y and the
    gradient d_r that reaches r by other ways.  dx is the gradient of x and of the residual alike; dweight and dbias are
    fp32."""
    return _native().layernorm_backward(dy, r, weight, d_r, eps, workspace)


# ---------------------------------------------------------------- gated norm of a recurrence's output

def _gate_code(gate):
    if gate not in ("silu", "sigmoid"):
        raise ValueError(f"gate: 'silu' or 'sigmoid' is needed, got {gate!r}")
    return 0 if gate == "silu" else 1


@_streamed
def gated_norm_forward(x, z, weight, *, gate="silu", eps=1e-6):
    """y = gated_norm_forward(x, z, weight): x / sqrt(mean(x^2) + eps) * weight * gate(z), the mean over the V columns of
    each head.  x, z [..., H, V] (slices of a wider token row are used in place); weight [V], or [H, V] for weights of
    each head; gate: "silu" or "sigmoid"."""
    return _native().gated_norm_forward(x, z, weight, _gate_code(gate), eps)


@_streamed
def gated_norm_backward(dy, x, z, weight, *, gate="silu", eps=1e-6, workspace=None):
    """dx, dz, dweight = gated_norm_backward(dy, x, z, weight): the gradient of gated_norm_forward's y, from its inputs.
    dweight is fp32, like weight."""
    return _native().gated_norm_backward(dy, x, z, weight, _gate_code(gate), eps, workspace)
