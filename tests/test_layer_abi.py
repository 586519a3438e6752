"""Host-side checks of the layer operators' C ABI: bad arguments are refused with the documented status codes before
anything is launched, and the workspace sizes follow from the problem alone (no GPU needed)."""
import ctypes

import pytest

from chunked_gated_delta_prepare_gb300 import build as gdr_build
from chunked_gated_delta_prepare_gb300 import gdr

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 5, 9


@pytest.fixture(scope="module")
def lib():
    gdr_build.build()
    return gdr.load()


def norm(**kw):
    return gdr.gdr_norm_problem(**(dict(rows=4, D=64, io_dtype=1, group=0, eps=1e-6) | kw))


def conv(**kw):
    return gdr.gdr_conv_problem(**(dict(n=2, T=8, total=16, D=64, pool=4, W=4, io_dtype=1, silu=1) | kw))


def ssm(**kw):
    return gdr.gdr_ssm_problem(**(dict(n=2, T=8, total=16, D=64, N=16, G=1, pool=4, io_dtype=1, softplus=1) | kw))


def step(**kw):
    return gdr.gdr_step_problem(**(dict(B=2, H=2, HV=4, K=64, V=64, pool=4, io_dtype=1, gate=0, scale=-1.0) | kw))


def call(name, p, ptrs):
    lib = gdr.load()
    return getattr(lib, name)(ctypes.byref(p) if p is not None else None, *ptrs)


# pointers that are never followed: each call is refused first
CALLS = {
    "gdr_norm_forward": (norm, dict(x=16, residual=16, w=16, y=16, r=16, y8=16, scales=16, stream=None)),
    "gdr_norm_backward": (norm, dict(dy=16, r=16, w=16, dr=16, dx=16, dw=16, ws=256, nbytes=1 << 30, stream=None)),
    "gdr_conv_forward": (conv, dict(cu=None, x=16, w=16, b=16, state=16, y=16, out=16, stream=None)),
    "gdr_conv_backward": (conv, dict(cu=None, x=16, w=16, b=16, state=16, dy=16, dout=16, dx=16, dw=16, db=16, dstate=16,
                                     ws=256, nbytes=1 << 30, stream=None)),
    "gdr_conv_step": (conv, dict(slots=None, x=16, w=16, b=16, state=16, y=16, stream=None)),
    "gdr_ssm_forward": (ssm, dict(cu=None, x=16, dt=16, A=16, B=16, C=16, Dk=16, z=16, bias=16, h0=16, y=16, h=16,
                                  ws=256, nbytes=1 << 30, stream=None)),
    "gdr_ssm_backward": (ssm, dict(cu=None, x=16, dt=16, A=16, B=16, C=16, Dk=16, z=16, bias=16, h0=16, dy=16, dh=16,
                                   dx=16, ddt=16, dA=16, dB=16, dC=16, dDk=16, dz=16, dbias=16, dh0=16, ws=256,
                                   nbytes=1 << 30, stream=None)),
    "gdr_ssm_step": (ssm, dict(slots=None, x=16, dt=16, A=16, B=16, C=16, Dk=16, z=16, bias=16, h=16, y=16,
                               stream=None)),
    "gdr_delta_step": (step, dict(slots=None, q=16, k=16, v=16, g=16, beta=16, h=16, o=16, stream=None)),
}
REQUIRED = {
    "gdr_norm_forward": ["x", "w"], "gdr_norm_backward": ["dy", "r", "w", "dx", "dw"],
    "gdr_conv_forward": ["x", "w", "y"], "gdr_conv_backward": ["x", "w", "dy", "dx", "dw", "db"],
    "gdr_conv_step": ["x", "w", "state", "y"], "gdr_ssm_forward": ["x", "dt", "A", "B", "C", "y"],
    "gdr_ssm_backward": ["x", "dt", "A", "B", "C", "dy", "dx", "ddt", "dA", "dB", "dC", "dz"],
    "gdr_ssm_step": ["x", "dt", "A", "B", "C", "h", "y"], "gdr_delta_step": ["q", "k", "v", "g", "beta", "h", "o"],
}


@pytest.mark.parametrize("name", CALLS)
def test_null_problem(lib, name):
    assert call(name, None, CALLS[name][1].values()) == NULL


@pytest.mark.parametrize("name,ptr", [(n, p) for n, ps in REQUIRED.items() for p in ps])
def test_null_required_pointer(lib, name, ptr):
    make, ptrs = CALLS[name]
    assert call(name, make(), (ptrs | {ptr: None}).values()) == NULL


@pytest.mark.parametrize("name,ptr", [(n, p) for n, (_, ps) in CALLS.items() for p in ps
                                      if p not in ("stream", "nbytes", "y8", "ws")])
def test_misaligned_pointer(lib, name, ptr):
    make, ptrs = CALLS[name]
    assert call(name, make(), (ptrs | {ptr: 17}).values()) == ALIGN


@pytest.mark.parametrize("name", [n for n, (_, p) in CALLS.items() if "ws" in p])
def test_workspace(lib, name):
    make, ptrs = CALLS[name]
    p = make(T=4000) if make is ssm else make()              # long enough for segments
    packed = [] if make is norm else [0]
    need = getattr(lib, name + "_workspace_bytes")(ctypes.byref(p), *packed)
    assert need > 0
    assert call(name, p, (ptrs | dict(ws=None)).values()) == WORKSPACE
    assert call(name, p, (ptrs | dict(nbytes=need - 1)).values()) == WORKSPACE
    assert call(name, p, (ptrs | dict(ws=128)).values()) == ALIGN
    assert getattr(lib, name + "_workspace_bytes")(None, *packed) == 0
    p.io_dtype = 7
    assert getattr(lib, name + "_workspace_bytes")(ctypes.byref(p), *packed) == 0


@pytest.mark.parametrize("name", CALLS)
def test_bad_dtype(lib, name):
    make, ptrs = CALLS[name]
    assert call(name, make(io_dtype=3), ptrs.values()) == DTYPE


@pytest.mark.parametrize("name,kw,status", [
    ("gdr_norm_forward", dict(rows=-1), SHAPE), ("gdr_norm_forward", dict(D=0), SHAPE),
    ("gdr_norm_forward", dict(D=32769), SHAPE), ("gdr_norm_forward", dict(x_ld=63), SHAPE),
    ("gdr_norm_forward", dict(group=16), ARG), ("gdr_norm_forward", dict(eps=float("nan")), ARG),
    ("gdr_norm_forward", dict(eps=float("inf")), ARG), ("gdr_norm_forward", dict(eps=-1e-6), ARG),
    ("gdr_conv_forward", dict(n=0), SHAPE), ("gdr_conv_forward", dict(T=0), SHAPE),
    ("gdr_conv_forward", dict(D=0), SHAPE), ("gdr_conv_forward", dict(W=1), SHAPE),
    ("gdr_conv_forward", dict(W=5), SHAPE), ("gdr_conv_forward", dict(silu=2), ARG),
    ("gdr_conv_forward", dict(n=1 << 20, T=1 << 12), SHAPE), ("gdr_conv_forward", dict(x_ld=10), SHAPE),
    ("gdr_conv_step", dict(n=5), SHAPE), ("gdr_conv_step", dict(pool=0), SHAPE),
    ("gdr_ssm_forward", dict(N=0), SHAPE), ("gdr_ssm_forward", dict(N=65), SHAPE),
    ("gdr_ssm_forward", dict(G=3), SHAPE), ("gdr_ssm_forward", dict(G=0), SHAPE),
    ("gdr_ssm_forward", dict(D=1 << 20, G=1 << 20), SHAPE), ("gdr_ssm_forward", dict(b_ld=15), SHAPE),
    ("gdr_ssm_forward", dict(softplus=-1), ARG), ("gdr_ssm_backward", dict(T=-4), SHAPE),
    ("gdr_ssm_step", dict(n=5), SHAPE), ("gdr_delta_step", dict(HV=3), SHAPE), ("gdr_delta_step", dict(B=5), SHAPE),
    ("gdr_delta_step", dict(K=32), SHAPE), ("gdr_delta_step", dict(V=96), SHAPE), ("gdr_delta_step", dict(H=0), SHAPE),
    ("gdr_delta_step", dict(gate=2), DTYPE), ("gdr_delta_step", dict(scale=float("inf")), ARG),
    ("gdr_delta_step", dict(q_ld=64), SHAPE),
])
def test_bad_problem(lib, name, kw, status):
    make, ptrs = CALLS[name]
    assert call(name, make(**kw), ptrs.values()) == status


def test_nothing_to_write_or_half_of_a_pair(lib):
    _, ptrs = CALLS["gdr_norm_forward"]
    none = dict(y=None, r=None, y8=None, scales=None)
    assert call("gdr_norm_forward", norm(), (ptrs | none).values()) == NULL
    assert call("gdr_norm_forward", norm(), (ptrs | dict(scales=None)).values()) == NULL
    assert call("gdr_norm_forward", norm(), (ptrs | dict(y8=None)).values()) == NULL


def test_no_rows_is_no_work(lib):
    assert call("gdr_norm_forward", norm(rows=0), [None] * 8) == 0


def test_the_binding_is_built_and_refuses_host_tensors(lib):
    import torch
    from chunked_gated_delta_prepare_gb300 import layer
    x, w = torch.zeros(2, 64), torch.zeros(64)
    for f in (lambda: layer.norm_forward(x, w), lambda: layer.norm_backward(x, x, w),
              lambda: layer.conv_forward(x[None], torch.zeros(64, 4)),
              lambda: layer.conv_step(x, torch.zeros(64, 4), None, torch.zeros(2, 3, 64)),
              lambda: layer.ssm_forward(x[None], x[None], torch.zeros(64, 16), torch.zeros(1, 2, 1, 16),
                                        torch.zeros(1, 2, 1, 16)),
              lambda: layer.delta_step(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), torch.zeros(1, 1, 64),
                                       torch.zeros(1, 1), torch.zeros(1, 1), torch.zeros(1, 1, 64, 64)),
              lambda: layer.norm_forward(None, w), lambda: layer.norm_forward([1.0], w)):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("name", ["gdr_ssm_forward", "gdr_ssm_backward", "gdr_ssm_step"])
def test_channels_beyond_the_grid(lib, name):
    """At more than 32 states a block has as few as 16 channels: 2^20 of them are one block more than a grid takes."""
    make, ptrs = CALLS[name]
    assert call(name, make(D=1 << 20, N=64, n=1, T=1), ptrs.values()) == SHAPE


@pytest.mark.parametrize("name", ["gdr_conv_forward", "gdr_ssm_forward", "gdr_norm_forward"])
def test_tokens_beyond_31_bit_tiles(lib, name):
    make, ptrs = CALLS[name]
    kw = dict(rows=1 << 30) if make is norm else dict(n=1 << 30, T=1)
    assert call(name, make(**kw), ptrs.values()) == SHAPE
    if make is not norm:
        packed = make(n=1, total=1 << 30)
        assert call(name, packed, (ptrs | dict(cu=16)).values()) == SHAPE
