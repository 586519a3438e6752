"""ctypes binding of libgdr's layer operators (include/gdr.h, "the layer around the recurrence").

    norm_forward, norm_backward               root-mean-square norm, residual, 8-bit output
    conv_forward, conv_backward, conv_step    short causal convolution
    ssm_forward, ssm_backward, ssm_step       selective state space scan
    delta_step                                the gated delta rule for one token

Argument marshalling only: the arithmetic runs in libgdr's CUDA kernels, and a missing library raises.  Each call
takes device tensors, allocates its outputs (and a workspace, unless one is given) and returns as soon as its kernels
are queued on the current stream, or on `stream`, to which the outputs and the workspace then belong.  Shapes, types
and devices that do not fit raise ValueError; what the library refuses raises GdrError.

Inputs of tokens may be slices of a wider projection ([T, D] or [B, T, D] views with contiguous columns and one
stride for all rows); views with other strides are copied first.  States are changed in place and must be contiguous.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

import torch

from .gdr import (DTYPES, _check, _ptr, gdr_conv_problem, gdr_norm_problem, gdr_ssm_problem, gdr_step_problem, load)


def _on(stream):
    """Allocations belong to the stream the kernels run on."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _stream(stream, t):
    """The stream's handle; the current one of the tensor's device without a stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.device.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _need(ok, text):
    if not ok:
        raise ValueError(text)


def _rows(t, dtype, shape, name):
    """The tensor (copied if its rows have no one stride) and its row stride for the C ABI (0: contiguous)."""
    if t is None:
        return None, 0
    _need(t.is_cuda and t.dtype == dtype and t.shape == shape,
          f"{name}: a device tensor {tuple(shape)} of {dtype} is needed, got {tuple(t.shape)} {t.dtype} on {t.device}")
    if t.is_contiguous():
        return t, 0
    cols = shape[-1]
    lead = [(n, st) for n, st in zip(shape[:-1], t.stride()[:-1]) if n != 1]
    ok = lead and (cols == 1 or t.stride(-1) == 1) and lead[-1][1] >= cols
    for (_, outer), (n, inner) in zip(lead[:-1], lead[1:]):
        ok = ok and outer == n * inner
    return (t, lead[-1][1]) if ok else (t.contiguous(), 0)


def _whole(t, dtype, shape, name):
    """A contiguous device tensor of this type and shape, or None."""
    if t is not None:
        _need(t.is_cuda and t.dtype == dtype and t.shape == shape and t.is_contiguous(),
              f"{name}: a contiguous device tensor {tuple(shape)} of {dtype} is needed, got {tuple(t.shape)} {t.dtype} "
              f"on {t.device}")
    return t


def _workspace(workspace, nbytes, device):
    """(tensor, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        workspace = torch.empty(nbytes, device=device, dtype=torch.uint8) if nbytes else None
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def _io(t):
    _need(t.dtype in DTYPES, f"io type {t.dtype}: float32, bfloat16 or float16 is needed")
    return DTYPES[t.dtype]


def _sequences(x, cu_seqlens):
    """(n, T, total) of x [B, T, D] or, with the device int32 cu_seqlens [n + 1], packed x [total, D]."""
    if cu_seqlens is None:
        _need(x.dim() == 3 and x.shape[0] > 0 and x.shape[1] > 0, f"x: [B, T, D] is needed, got {tuple(x.shape)}")
        return x.shape[0], x.shape[1], 0
    _need(x.dim() == 2, f"x: packed tokens [total, D] are needed with cu_seqlens, got {tuple(x.shape)}")
    _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2, "cu_seqlens: [n + 1] entries are needed")
    _whole(cu_seqlens, torch.int32, cu_seqlens.shape, "cu_seqlens")
    return cu_seqlens.numel() - 1, 0, x.shape[0]


# ---------------------------------------------------------------- root-mean-square norm

def norm_forward(x, weight, residual=None, *, eps=1e-6, quant=None, want_y=True, stream=None):
    """y, r, y8, scales = norm_forward(x, weight, residual): the norm of s = x + residual over the last dimension.

    y = s * weight / sqrt(mean(s^2) + eps) in x's type (None with want_y=False); r = s in x's type, the new residual
    (x itself without a residual).  quant: None, "row" or a group of 32, 64 or 128 columns; then y8 is y / scale in
    float8_e4m3fn and scales fp32 holds one scale a row [..., 1] or a group [..., ceil(D / group)].
    """
    io, shape = _io(x), x.shape
    D = shape[-1]
    _need(quant is None or quant == "row" or (isinstance(quant, int) and quant > 0), f"quant: {quant!r}")
    x, x_ld = _rows(x, x.dtype, shape, "x")
    residual, res_ld = _rows(residual, x.dtype, shape, "residual")
    _whole(weight, x.dtype, (D,), "weight")
    group = 0 if quant in (None, "row") else quant
    rows = x.numel() // D if D else 0
    p = gdr_norm_problem(rows, D, x_ld, res_ld, io, group, eps)
    with _on(stream):
        y = torch.empty(shape, device=x.device, dtype=x.dtype) if want_y else None
        r = torch.empty(shape, device=x.device, dtype=x.dtype) if residual is not None else None
        y8 = scales = None
        if quant is not None:
            y8 = torch.empty(shape, device=x.device, dtype=torch.float8_e4m3fn)
            scales = torch.empty(*shape[:-1], -(-D // group) if group else 1, device=x.device, dtype=torch.float32)
        _check(load().gdr_norm_forward(ctypes.byref(p), _ptr(x), _ptr(residual), _ptr(weight), _ptr(y), _ptr(r),
                                       _ptr(y8), _ptr(scales), _stream(stream, x)), "gdr_norm_forward")
    return y, x if r is None else r, y8, scales


def norm_backward(dy, r, weight, d_r=None, *, eps=1e-6, workspace=None, stream=None):
    """dx, dweight = norm_backward(dy, r, weight, d_r): from the forward's r, the gradient dy of y and the gradient d_r
    that reaches r by other ways.  dx is the gradient of x and of the residual alike; dweight is fp32."""
    D = r.shape[-1]
    r, dy = r.contiguous(), dy.contiguous()
    d_r = d_r.contiguous() if d_r is not None else None
    for t, name in ((r, "r"), (dy, "dy"), (d_r, "d_r")):
        _whole(t, r.dtype, r.shape, name)
    _whole(weight, r.dtype, (D,), "weight")
    p = gdr_norm_problem(r.numel() // D if D else 0, D, 0, 0, _io(r), 0, eps)
    with _on(stream):
        dx, dw = torch.empty_like(r), torch.empty(D, device=r.device, dtype=torch.float32)
        ws, have = _workspace(workspace, load().gdr_norm_backward_workspace_bytes(ctypes.byref(p)), r.device)
        _check(load().gdr_norm_backward(ctypes.byref(p), _ptr(dy), _ptr(r), _ptr(weight), _ptr(d_r), _ptr(dx), _ptr(dw),
                                        _ptr(ws), have, _stream(stream, r)), "gdr_norm_backward")
    return dx, dw


# ---------------------------------------------------------------- short causal convolution

def _conv(x, weight, bias, cu_seqlens, silu):
    io, D = _io(x), x.shape[-1]
    _need(weight.dim() == 2, "weight: [D, W] is needed")
    _whole(weight, x.dtype, (D, weight.shape[1]), "weight")
    _whole(bias, x.dtype, (D,), "bias")
    n, T, total = _sequences(x, cu_seqlens)
    x, ld = _rows(x, x.dtype, x.shape, "x")
    return x, gdr_conv_problem(n, T, total, D, ld, 0, weight.shape[1], io, bool(silu))


def conv_forward(x, weight, bias=None, state=None, *, silu=True, cu_seqlens=None, want_state=True, stream=None):
    """y, state_out = conv_forward(x, weight, bias, state): each channel's tokens with the W taps of its weight row.

    x [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); weight [D, W] (W = 2, 3 or 4) and bias
    [D] in x's type; state [n, W - 1, D]: the inputs before the first token, oldest first (None: zero).  state_out has
    the last W - 1 inputs of each sequence (None with want_state=False)."""
    x, p = _conv(x, weight, bias, cu_seqlens, silu)
    states = (p.n, p.W - 1, p.D)
    _whole(state, x.dtype, states, "state")
    with _on(stream):
        y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
        out = torch.empty(states, device=x.device, dtype=x.dtype) if want_state else None
        _check(load().gdr_conv_forward(ctypes.byref(p), _ptr(cu_seqlens), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state),
                                       _ptr(y), _ptr(out), _stream(stream, x)), "gdr_conv_forward")
    return y, out


def conv_backward(x, weight, bias, dy, state=None, d_state_out=None, *, silu=True, cu_seqlens=None, workspace=None,
                  stream=None):
    """dx, dweight, dbias, dstate = conv_backward(x, weight, bias, dy, state, d_state_out): the gradient of
    conv_forward's y and state_out (d_state_out None: unused).  dweight and dbias are fp32; dbias is None without a
    bias, dstate without a state."""
    x, p = _conv(x, weight, bias, cu_seqlens, silu)
    states = (p.n, p.W - 1, p.D)
    _whole(state, x.dtype, states, "state")
    dy = _whole(dy.contiguous(), x.dtype, x.shape, "dy")
    if d_state_out is not None:
        d_state_out = _whole(d_state_out.contiguous(), x.dtype, states, "d_state_out")
    with _on(stream):
        dx = torch.empty(x.shape, device=x.device, dtype=x.dtype)
        dw = torch.empty(p.D, p.W, device=x.device, dtype=torch.float32)
        db = torch.empty(p.D, device=x.device, dtype=torch.float32)
        dstate = torch.empty_like(state) if state is not None else None
        need = load().gdr_conv_backward_workspace_bytes(ctypes.byref(p), cu_seqlens is not None)
        ws, have = _workspace(workspace, need, x.device)
        _check(load().gdr_conv_backward(ctypes.byref(p), _ptr(cu_seqlens), _ptr(x), _ptr(weight), _ptr(bias),
                                        _ptr(state), _ptr(dy), _ptr(d_state_out), _ptr(dx), _ptr(dw), _ptr(db),
                                        _ptr(dstate), _ptr(ws), have, _stream(stream, x)), "gdr_conv_backward")
    return dx, dw, db if bias is not None else None, dstate


def conv_step(x, weight, bias, state, *, silu=True, slots=None, stream=None):
    """y = conv_step(x, weight, bias, state): one token x [n, D] of n sequences.  state [pool, W - 1, D] is shifted in
    place, row i using state slots[i] (device int32; None: state i); a slot outside the pool marks a padding row."""
    io, D = _io(x), x.shape[-1]
    _need(x.dim() == 2 and weight.dim() == 2 and state.dim() == 3, "x [n, D], weight [D, W], state [pool, W - 1, D]")
    _whole(weight, x.dtype, (D, weight.shape[1]), "weight")
    _whole(bias, x.dtype, (D,), "bias")
    _whole(state, x.dtype, (state.shape[0], weight.shape[1] - 1, D), "state")
    _whole(slots, torch.int32, x.shape[:1], "slots")
    x, ld = _rows(x, x.dtype, x.shape, "x")
    p = gdr_conv_problem(x.shape[0], 1, 0, D, ld, state.shape[0], weight.shape[1], io, bool(silu))
    with _on(stream):
        y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
        _check(load().gdr_conv_step(ctypes.byref(p), _ptr(slots), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state),
                                    _ptr(y), _stream(stream, x)), "gdr_conv_step")
    return y


# ---------------------------------------------------------------- selective state space scan

def _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, T, total, pool):
    """The problem, and its tensors in the C ABI's order (x, dt, A, B, C, D, z, dt_bias)."""
    io, shape, ch = _io(x), x.shape, x.shape[-1]
    _need(A.dim() == 2 and B.dim() == x.dim() + 1, "A [D, N] and B [..., G, N] are needed")
    G, N = B.shape[-2:]
    x, x_ld = _rows(x, x.dtype, shape, "x")
    dt, dt_ld = _rows(dt, x.dtype, shape, "dt")
    z, z_ld = _rows(z, x.dtype, shape, "z")
    bc = (*shape[:-1], G * N)
    _need(C.shape == B.shape, f"C: {tuple(B.shape)} is needed, got {tuple(C.shape)}")
    B, b_ld = _rows(B.flatten(-2), x.dtype, bc, "B")
    C, c_ld = _rows(C.flatten(-2), x.dtype, bc, "C")
    _whole(A, torch.float32, (ch, N), "A")
    _whole(D, torch.float32, (ch,), "D")
    _whole(dt_bias, torch.float32, (ch,), "dt_bias")
    p = gdr_ssm_problem(n, T, total, ch, N, G, x_ld, dt_ld, z_ld, b_ld, c_ld, pool, io, bool(softplus))
    return p, (x, dt, A, B, C, D, z, dt_bias)


def ssm_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True, cu_seqlens=None,
                want_h_final=True, workspace=None, stream=None):
    """y, h_final = ssm_forward(x, dt, A, B, C, D, z, dt_bias, h0): the selective state space scan.

    x, dt, z [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); B, C [..., G, N], the D / G channels
    of a group sharing one; A [D, N], D [D], dt_bias [D] fp32; h0 [n, D, N] fp32 (None: zero).
        Delta = softplus(dt + dt_bias);  h = exp(Delta A) h + Delta x B;  y = (C.h + D x) silu(z)
    y is in the io type, h_final [n, D, N] fp32 (None with want_h_final=False)."""
    n, T, total = _sequences(x, cu_seqlens)
    p, tensors = _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, T, total, 0)
    states = (n, p.D, p.N)
    _whole(h0, torch.float32, states, "h0")
    with _on(stream):
        y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
        h = torch.empty(states, device=x.device, dtype=torch.float32) if want_h_final else None
        ws, have = _workspace(workspace, load().gdr_ssm_forward_workspace_bytes(ctypes.byref(p), cu_seqlens is not None),
                              x.device)
        _check(load().gdr_ssm_forward(ctypes.byref(p), _ptr(cu_seqlens), *map(_ptr, tensors), _ptr(h0), _ptr(y), _ptr(h),
                                      _ptr(ws), have, _stream(stream, x)), "gdr_ssm_forward")
    return y, h


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


def ssm_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, h0=None, dh_final=None, *, softplus=True,
                 cu_seqlens=None, workspace=None, stream=None) -> SsmGrads:
    """The gradient of ssm_forward's y and h_final (dh_final None: unused), from the forward's inputs alone.  dx, ddt, dB,
    dC, dz are in the io type, the others fp32; those of inputs that are None are None."""
    n, T, total = _sequences(x, cu_seqlens)
    p, tensors = _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, T, total, 0)
    states, bc, io = (n, p.D, p.N), B.shape, x.dtype
    _whole(h0, torch.float32, states, "h0")
    dy = _whole(dy.contiguous(), io, x.shape, "dy")
    if dh_final is not None:
        dh_final = _whole(dh_final.contiguous(), torch.float32, states, "dh_final")
    with _on(stream):
        dx, ddt = (torch.empty(x.shape, device=x.device, dtype=io) for _ in range(2))
        dz = torch.empty(x.shape, device=x.device, dtype=io) if z is not None else None
        dB, dC = (torch.empty(bc, device=x.device, dtype=io) for _ in range(2))
        dA = torch.empty_like(A)
        dD, dbias, dh0 = (torch.empty_like(t) if t is not None else None for t in (D, dt_bias, h0))
        need = load().gdr_ssm_backward_workspace_bytes(ctypes.byref(p), cu_seqlens is not None)
        ws, have = _workspace(workspace, need, x.device)
        _check(load().gdr_ssm_backward(ctypes.byref(p), _ptr(cu_seqlens), *map(_ptr, tensors), _ptr(h0), _ptr(dy),
                                       _ptr(dh_final), _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD),
                                       _ptr(dz), _ptr(dbias), _ptr(dh0), _ptr(ws), have, _stream(stream, x)),
               "gdr_ssm_backward")
    return SsmGrads(dx, ddt, dA, dB, dC, dD, dz, dbias, dh0)


def ssm_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, softplus=True, slots=None, stream=None):
    """y = ssm_step(x, dt, A, B, C, h, D, z, dt_bias): one token of n rows, x, dt, z [n, D], B, C [n, G, N].  h [pool, D,
    N] fp32 is changed in place, row i using state slots[i] (device int32; None: state i); a slot outside the pool marks
    a padding row, whose y is zero."""
    _need(x.dim() == 2 and h.dim() == 3, "x [n, D], h [pool, D, N]")
    p, tensors = _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, x.shape[0], 1, 0, h.shape[0])
    _whole(h, torch.float32, (h.shape[0], p.D, p.N), "h")
    _whole(slots, torch.int32, x.shape[:1], "slots")
    with _on(stream):
        y = torch.empty(x.shape, device=x.device, dtype=x.dtype)
        _check(load().gdr_ssm_step(ctypes.byref(p), _ptr(slots), *map(_ptr, tensors), _ptr(h), _ptr(y),
                                   _stream(stream, x)), "gdr_ssm_step")
    return y


# ---------------------------------------------------------------- the gated delta rule, one token

def delta_step(q, k, v, g, beta, h, *, scale=None, slots=None, stream=None):
    """o = delta_step(q, k, v, g, beta, h): one token of B rows, as forward() computes it for T = 1.

    q, k [B, H, K], v [B, HV, V] (slices of a wider [B, ...] row are used in place), beta [B, HV] in the io type;
    g [B, HV] or [B, HV, K] fp32.  h [pool, HV, K, V] fp32 is changed in place, row i using state slots[i] (device
    int32; None: state i); a slot outside the pool marks a padding row, whose o is zero."""
    _need(q.dim() == 3 and v.dim() == 3 and h.dim() == 4, "q [B, H, K], v [B, HV, V], h [pool, HV, K, V]")
    (B, H, K), (_, HV, V) = q.shape, v.shape
    io = _io(q)
    flat = []
    for t, cols, name in ((q, H * K, "q"), (k, H * K, "k"), (v, HV * V, "v")):
        _need(t.dim() == 3 and t.shape[0] == B, f"{name}: [B, heads, dim] is needed")
        flat += _rows(t.flatten(1), q.dtype, (B, cols), name)
    q, q_ld, k, k_ld, v, v_ld = flat
    per_k = g.dim() == 3
    _whole(g, torch.float32, (B, HV, K) if per_k else (B, HV), "g")
    _whole(beta, q.dtype, (B, HV), "beta")
    _whole(h, torch.float32, (h.shape[0], HV, K, V), "h")
    _whole(slots, torch.int32, (B,), "slots")
    p = gdr_step_problem(B, H, HV, K, V, h.shape[0], q_ld, k_ld, v_ld, io, per_k, -1.0 if scale is None else scale)
    with _on(stream):
        o = torch.empty(B, HV, V, device=q.device, dtype=q.dtype)
        _check(load().gdr_delta_step(ctypes.byref(p), _ptr(slots), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                     _ptr(h), _ptr(o), _stream(stream, q)), "gdr_delta_step")
    return o
