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

A single-token call takes some 10 microseconds of host time beside a kernel of a few, so the checks below are written
for speed: one condition a tensor, and no text before something is wrong.
"""
from __future__ import annotations

import functools
from ctypes import byref
from typing import NamedTuple

import torch

from .gdr import (DTYPES, GDR_OK, GdrError, gdr_conv_problem, gdr_norm_problem, gdr_ssm_problem, gdr_step_problem, load)

_current_stream = torch._C._cuda_getCurrentRawStream
F32, I32 = torch.float32, torch.int32


def _streamed(f):
    """Adds `stream` to a call: allocations and kernels of the call then belong to that stream."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
            return f(*args, **kw)
    return call


def _run(name, *args):
    status = getattr(load(), name)(*args)
    if status != GDR_OK:
        raise GdrError(status, name)


def _refuse(t, dtype, shape, name, what=""):
    got = f"{tuple(t.shape)} {t.dtype} on {t.device}" if isinstance(t, torch.Tensor) else repr(t)
    raise ValueError(f"{name}: a {what}device tensor {tuple(shape)} of {dtype} is needed, got {got}")


def _rows(t, dtype, shape, name):
    """The tensor (copied if its rows have no one stride) and its row stride for the C ABI (0: contiguous)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        _refuse(t, dtype, shape, name)
    if t.is_contiguous():
        return t, 0
    strides, cols = t.stride(), shape[-1]
    if strides[-1] == 1 or cols == 1:
        if len(strides) == 2 and strides[0] >= cols:
            return t, strides[0]
        lead = [(n, st) for n, st in zip(shape[:-1], strides) if n != 1]
        if lead and lead[-1][1] >= cols and all(a[1] == b[0] * b[1] for a, b in zip(lead, lead[1:])):
            return t, lead[-1][1]
    return t.contiguous(), 0


def _heads(t, dtype, shape, name):
    """_rows of a tensor whose last two dimensions make up a row's columns."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        _refuse(t, dtype, shape, name)
    if t.is_contiguous():
        return t, 0
    if len(shape) == 3:
        row, head, one = t.stride()
        if one == 1 and (head == shape[2] or shape[1] == 1) and row >= shape[1] * shape[2]:
            return t, row
    flat = t.flatten(-2)                   # a view where the columns are contiguous, else a copy
    return _rows(flat, dtype, flat.shape, name)


def _whole(t, dtype, shape, name):
    """The address of a contiguous device tensor of this type and shape; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(t, dtype, shape, name, "contiguous ")
    return t.data_ptr()


def _at(t):
    return 0 if t is None else t.data_ptr()


def _workspace(workspace, nbytes, device):
    """(tensor, bytes) of the caller's workspace, or of a new one."""
    if workspace is None:
        if not nbytes:
            return None, 0
        return torch.empty(nbytes, device=device, dtype=torch.uint8), nbytes
    return workspace, workspace.numel() * workspace.element_size()


def _io(dtype):
    io = DTYPES.get(dtype)
    if io is None:
        raise ValueError(f"io type {dtype}: float32, bfloat16 or float16 is needed")
    return io


def _sequences(x, cu_seqlens):
    """(n, T, total) of x [B, T, D] or, with the device int32 cu_seqlens [n + 1], packed x [total, D]."""
    if cu_seqlens is None:
        if x.dim() != 3 or x.shape[0] < 1 or x.shape[1] < 1:
            raise ValueError(f"x: [B, T, D] is needed, got {tuple(x.shape)}")
        return x.shape[0], x.shape[1], 0
    if x.dim() != 2:
        raise ValueError(f"x: packed tokens [total, D] are needed with cu_seqlens, got {tuple(x.shape)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens: [n + 1] entries are needed")
    _whole(cu_seqlens, I32, cu_seqlens.shape, "cu_seqlens")
    return cu_seqlens.numel() - 1, 0, x.shape[0]


# ---------------------------------------------------------------- root-mean-square norm

@_streamed
def norm_forward(x, weight, residual=None, *, eps=1e-6, quant=None, want_y=True):
    """y, r, y8, scales = norm_forward(x, weight, residual): the norm of s = x + residual over the last dimension.

    y = s * weight / sqrt(mean(s^2) + eps) in x's type (None with want_y=False); r = s in x's type, the new residual
    (x itself without a residual).  quant: None, "row" or a group of 32, 64 or 128 columns; then y8 is y / scale in
    float8_e4m3fn and scales fp32 holds one scale a row [..., 1] or a group [..., ceil(D / group)].
    """
    dtype, shape, device = x.dtype, x.shape, x.device
    D = shape[-1]
    if quant is None or quant == "row":
        group = 0
    elif isinstance(quant, int) and quant > 0:
        group = quant
    else:
        raise ValueError(f"quant: None, 'row' or a number of columns is needed, got {quant!r}")
    r = None
    src, x_ld = _rows(x, dtype, shape, "x")
    res, res_ld = _rows(residual, dtype, shape, "residual")
    w = _whole(weight, dtype, (D,), "weight")
    p = gdr_norm_problem(x.numel() // D if D else 0, D, x_ld, res_ld, _io(dtype), group, eps)
    y = torch.empty(shape, device=device, dtype=dtype) if want_y else None
    if res is not None:
        r = torch.empty(shape, device=device, dtype=dtype)
    y8 = scales = None
    if quant is not None:
        y8 = torch.empty(shape, device=device, dtype=torch.float8_e4m3fn)
        scales = torch.empty((*shape[:-1], -(-D // group) if group else 1), device=device, dtype=F32)
    _run("gdr_norm_forward", byref(p), src.data_ptr(), _at(res), w, _at(y), _at(r), _at(y8), _at(scales),
         _current_stream(device.index))
    return y, x if r is None else r, y8, scales


@_streamed
def norm_backward(dy, r, weight, d_r=None, *, eps=1e-6, workspace=None):
    """dx, dweight = norm_backward(dy, r, weight, d_r): from the forward's r, the gradient dy of y and the gradient d_r
    that reaches r by other ways.  dx is the gradient of x and of the residual alike; dweight is fp32."""
    dtype, shape, device = r.dtype, r.shape, r.device
    D = shape[-1]
    r, dy = r.contiguous(), dy.contiguous()
    d_r = d_r.contiguous() if d_r is not None else None
    ptrs = [_whole(dy, dtype, shape, "dy"), _whole(r, dtype, shape, "r"), _whole(weight, dtype, (D,), "weight"),
            _whole(d_r, dtype, shape, "d_r")]
    p = gdr_norm_problem(r.numel() // D if D else 0, D, 0, 0, _io(dtype), 0, eps)
    dx, dw = torch.empty_like(r), torch.empty(D, device=device, dtype=F32)
    ws, have = _workspace(workspace, load().gdr_norm_backward_workspace_bytes(byref(p)), device)
    _run("gdr_norm_backward", byref(p), *ptrs, dx.data_ptr(), dw.data_ptr(), _at(ws), have, _current_stream(device.index))
    return dx, dw


# ---------------------------------------------------------------- short causal convolution

def _conv(x, weight, bias, cu_seqlens, silu):
    """x (copied if need be), the problem, and the addresses of x, weight and bias."""
    dtype, D = x.dtype, x.shape[-1]
    if weight.dim() != 2:
        raise ValueError(f"weight: [D, W] is needed, got {tuple(weight.shape)}")
    W = weight.shape[1]
    w, b = _whole(weight, dtype, (D, W), "weight"), _whole(bias, dtype, (D,), "bias")
    n, T, total = _sequences(x, cu_seqlens)
    x, ld = _rows(x, dtype, x.shape, "x")
    return x, gdr_conv_problem(n, T, total, D, ld, 0, W, _io(dtype), bool(silu)), (x.data_ptr(), w, b)


@_streamed
def conv_forward(x, weight, bias=None, state=None, *, silu=True, cu_seqlens=None, want_state=True):
    """y, state_out = conv_forward(x, weight, bias, state): each channel's tokens with the W taps of its weight row.

    x [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); weight [D, W] (W = 2, 3 or 4) and bias
    [D] in x's type; state [n, W - 1, D]: the inputs before the first token, oldest first (None: zero).  state_out has
    the last W - 1 inputs of each sequence (None with want_state=False)."""
    x, p, ptrs = _conv(x, weight, bias, cu_seqlens, silu)
    dtype, device, states = x.dtype, x.device, (p.n, p.W - 1, p.D)
    state = _whole(state, dtype, states, "state")
    y = torch.empty(x.shape, device=device, dtype=dtype)
    out = torch.empty(states, device=device, dtype=dtype) if want_state else None
    _run("gdr_conv_forward", byref(p), _at(cu_seqlens), *ptrs, state, y.data_ptr(), _at(out),
         _current_stream(device.index))
    return y, out


@_streamed
def conv_backward(x, weight, bias, dy, state=None, d_state_out=None, *, silu=True, cu_seqlens=None, workspace=None):
    """dx, dweight, dbias, dstate = conv_backward(x, weight, bias, dy, state, d_state_out): the gradient of
    conv_forward's y and state_out (d_state_out None: unused).  dweight and dbias are fp32; dbias is None without a
    bias, dstate without a state."""
    x, p, ptrs = _conv(x, weight, bias, cu_seqlens, silu)
    dtype, device, states = x.dtype, x.device, (p.n, p.W - 1, p.D)
    state_at = _whole(state, dtype, states, "state")
    dy = dy.contiguous()
    dy_at = _whole(dy, dtype, x.shape, "dy")
    d_state_out = d_state_out.contiguous() if d_state_out is not None else None
    out_at = _whole(d_state_out, dtype, states, "d_state_out")
    dx = torch.empty(x.shape, device=device, dtype=dtype)
    dw = torch.empty(weight.shape, device=device, dtype=F32)
    db = torch.empty(p.D, device=device, dtype=F32)
    dstate = torch.empty_like(state) if state is not None else None
    need = load().gdr_conv_backward_workspace_bytes(byref(p), cu_seqlens is not None)
    ws, have = _workspace(workspace, need, device)
    _run("gdr_conv_backward", byref(p), _at(cu_seqlens), *ptrs, state_at, dy_at, out_at, dx.data_ptr(), dw.data_ptr(),
         db.data_ptr(), _at(dstate), _at(ws), have, _current_stream(device.index))
    return dx, dw, db if bias is not None else None, dstate


@_streamed
def conv_step(x, weight, bias, state, *, silu=True, slots=None):
    """y = conv_step(x, weight, bias, state): one token x [n, D] of n sequences.  state [pool, W - 1, D] is shifted in
    place, row i using state slots[i] (device int32; None: state i); a slot outside the pool marks a padding row."""
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x [n, D], weight [D, W] and state [pool, W - 1, D] are needed")
    dtype, shape, device = x.dtype, x.shape, x.device
    n, D = shape
    pool, W = state.shape[0], weight.shape[1]
    x, ld = _rows(x, dtype, shape, "x")
    p = gdr_conv_problem(n, 1, 0, D, ld, pool, W, _io(dtype), bool(silu))
    y = torch.empty(shape, device=device, dtype=dtype)
    _run("gdr_conv_step", byref(p), _whole(slots, I32, (n,), "slots"), x.data_ptr(),
         _whole(weight, dtype, (D, W), "weight"), _whole(bias, dtype, (D,), "bias"),
         _whole(state, dtype, (pool, W - 1, D), "state"), y.data_ptr(), _current_stream(device.index))
    return y


# ---------------------------------------------------------------- selective state space scan

def _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, T, total, pool):
    """The problem, the tensors behind its addresses (copies among them), and the addresses of x .. dt_bias in the C
    ABI's order."""
    dtype, shape = x.dtype, x.shape
    if A.dim() != 2 or B.dim() != len(shape) + 1:
        raise ValueError("A [D, N] and B [..., G, N] are needed")
    ch, bc = shape[-1], B.shape
    G, N = bc[-2:]
    if bc[:-2] != shape[:-1]:
        _refuse(B, dtype, (*shape[:-1], G, N), "B")
    x, x_ld = _rows(x, dtype, shape, "x")
    dt, dt_ld = _rows(dt, dtype, shape, "dt")
    z, z_ld = _rows(z, dtype, shape, "z")
    B, b_ld = _heads(B, dtype, bc, "B")
    C, c_ld = _heads(C, dtype, bc, "C")
    p = gdr_ssm_problem(n, T, total, ch, N, G, x_ld, dt_ld, z_ld, b_ld, c_ld, pool, _io(dtype), bool(softplus))
    return p, (x, dt, z, B, C), (x.data_ptr(), dt.data_ptr(), _whole(A, F32, (ch, N), "A"), B.data_ptr(), C.data_ptr(),
                                 _whole(D, F32, (ch,), "D"), _at(z), _whole(dt_bias, F32, (ch,), "dt_bias"))


@_streamed
def ssm_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, *, softplus=True, cu_seqlens=None,
                want_h_final=True, workspace=None):
    """y, h_final = ssm_forward(x, dt, A, B, C, D, z, dt_bias, h0): the selective state space scan.

    x, dt, z [B, T, D], or packed [total, D] with cu_seqlens (device int32 [n + 1]); B, C [..., G, N], the D / G channels
    of a group sharing one; A [D, N], D [D], dt_bias [D] fp32; h0 [n, D, N] fp32 (None: zero).
        Delta = softplus(dt + dt_bias);  h = exp(Delta A) h + Delta x B;  y = (C.h + D x) silu(z)
    y is in the io type, h_final [n, D, N] fp32 (None with want_h_final=False)."""
    n, T, total = _sequences(x, cu_seqlens)
    p, kept, ptrs = _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, T, total, 0)
    device, states = x.device, (n, p.D, p.N)
    h0 = _whole(h0, F32, states, "h0")
    y = torch.empty(x.shape, device=device, dtype=x.dtype)
    h = torch.empty(states, device=device, dtype=F32) if want_h_final else None
    ws, have = _workspace(workspace, load().gdr_ssm_forward_workspace_bytes(byref(p), cu_seqlens is not None), device)
    _run("gdr_ssm_forward", byref(p), _at(cu_seqlens), *ptrs, h0, y.data_ptr(), _at(h), _at(ws), have,
         _current_stream(device.index))
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


@_streamed
def ssm_backward(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, h0=None, dh_final=None, *, softplus=True,
                 cu_seqlens=None, workspace=None) -> SsmGrads:
    """The gradient of ssm_forward's y and h_final (dh_final None: unused), from the forward's inputs alone.  dx, ddt, dB,
    dC, dz are in the io type, the others fp32; those of inputs that are None are None."""
    n, T, total = _sequences(x, cu_seqlens)
    p, kept, ptrs = _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, T, total, 0)
    device, states, bc, io = x.device, (n, p.D, p.N), B.shape, x.dtype
    h0_at = _whole(h0, F32, states, "h0")
    dy = dy.contiguous()
    dy_at = _whole(dy, io, x.shape, "dy")
    dh_final = dh_final.contiguous() if dh_final is not None else None
    dh_at = _whole(dh_final, F32, states, "dh_final")
    dx, ddt = (torch.empty(x.shape, device=device, dtype=io) for _ in range(2))
    dz = torch.empty(x.shape, device=device, dtype=io) if z is not None else None
    dB, dC = (torch.empty(bc, device=device, dtype=io) for _ in range(2))
    dA = torch.empty_like(A)
    dD, dbias, dh0 = (torch.empty_like(t) if t is not None else None for t in (D, dt_bias, h0))
    ws, have = _workspace(workspace, load().gdr_ssm_backward_workspace_bytes(byref(p), cu_seqlens is not None), device)
    _run("gdr_ssm_backward", byref(p), _at(cu_seqlens), *ptrs, h0_at, dy_at, dh_at, dx.data_ptr(), ddt.data_ptr(),
         dA.data_ptr(), dB.data_ptr(), dC.data_ptr(), _at(dD), _at(dz), _at(dbias), _at(dh0), _at(ws), have,
         _current_stream(device.index))
    return SsmGrads(dx, ddt, dA, dB, dC, dD, dz, dbias, dh0)


@_streamed
def ssm_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, *, softplus=True, slots=None):
    """y = ssm_step(x, dt, A, B, C, h, D, z, dt_bias): one token of n rows, x, dt, z [n, D], B, C [n, G, N].  h [pool, D,
    N] fp32 is changed in place, row i using state slots[i] (device int32; None: state i); a slot outside the pool marks
    a padding row, whose y is zero."""
    if x.dim() != 2 or h.dim() != 3:
        raise ValueError("x [n, D] and h [pool, D, N] are needed")
    n, pool, device = x.shape[0], h.shape[0], x.device
    p, kept, ptrs = _ssm(x, dt, A, B, C, D, z, dt_bias, softplus, n, 1, 0, pool)
    h = _whole(h, F32, (pool, p.D, p.N), "h")
    y = torch.empty(x.shape, device=device, dtype=x.dtype)
    _run("gdr_ssm_step", byref(p), _whole(slots, I32, (n,), "slots"), *ptrs, h, y.data_ptr(),
         _current_stream(device.index))
    return y


# ---------------------------------------------------------------- the gated delta rule, one token

@_streamed
def delta_step(q, k, v, g, beta, h, *, scale=None, slots=None):
    """o = delta_step(q, k, v, g, beta, h): one token of B rows, as forward() computes it for T = 1.

    q, k [B, H, K], v [B, HV, V] (slices of a wider [B, ...] row are used in place), beta [B, HV] in the io type;
    g [B, HV] or [B, HV, K] fp32.  h [pool, HV, K, V] fp32 is changed in place, row i using state slots[i] (device
    int32; None: state i); a slot outside the pool marks a padding row, whose o is zero."""
    if q.dim() != 3 or v.dim() != 3 or h.dim() != 4:
        raise ValueError("q [B, H, K], v [B, HV, V] and h [pool, HV, K, V] are needed")
    dtype, device = q.dtype, q.device
    (B, H, K), (_, HV, V), pool = q.shape, v.shape, h.shape[0]
    q, q_ld = _heads(q, dtype, (B, H, K), "q")
    k, k_ld = _heads(k, dtype, (B, H, K), "k")
    v, v_ld = _heads(v, dtype, (B, HV, V), "v")
    per_k = g.dim() == 3
    p = gdr_step_problem(B, H, HV, K, V, pool, q_ld, k_ld, v_ld, _io(dtype), per_k, -1.0 if scale is None else scale)
    o = torch.empty((B, HV, V), device=device, dtype=dtype)
    _run("gdr_delta_step", byref(p), _whole(slots, I32, (B,), "slots"), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         _whole(g, F32, (B, HV, K) if per_k else (B, HV), "g"), _whole(beta, dtype, (B, HV), "beta"),
         _whole(h, F32, (pool, HV, K, V), "h"), o.data_ptr(), _current_stream(device.index))
    return o
