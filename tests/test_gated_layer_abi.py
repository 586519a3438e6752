"""Host-side checks of the C ABI of the gated linear recurrence, the layer norm and the gated norm: bad arguments are refused
with the documented status codes before anything is launched (no GPU needed)."""
import ctypes

import pytest

from chunked_gated_delta_prepare_gb300 import build as gdr_build
from chunked_gated_delta_prepare_gb300 import gdr

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 5, 9


@pytest.fixture(scope="module")
def lib():
    gdr_build.build()
    return gdr.load()


def lru(**kw):
    return gdr.gdr_lru_problem(**(dict(n=2, T=500, total=1000, D=64, pool=4, io_dtype=1, c=8.0) | kw))


def ln(**kw):
    return gdr.gdr_layernorm_problem(**(dict(rows=4, D=64, io_dtype=1, eps=1e-5) | kw))


def gn(**kw):
    return gdr.gdr_gated_norm_problem(**(dict(tokens=4, H=2, V=64, io_dtype=1, gate=0, per_head=0, eps=1e-6) | kw))


def call(name, p, ptrs):
    return getattr(gdr.load(), name)(ctypes.byref(p) if p is not None else None, *ptrs)


# pointers that are never followed: each call is refused first
CALLS = {
    "gdr_lru_forward": (lru, dict(cu=None, x=16, r=16, i=16, lam=16, h0=16, y=16, h=16, kept=16, ws=256, nbytes=1 << 30,
                                  stream=None)),
    "gdr_lru_backward": (lru, dict(cu=None, x=16, r=16, i=16, lam=16, h0=16, dy=16, dh=16, kept=16, dx=16, dr=16, di=16,
                                   dlam=16, dh0=16, ws=256, nbytes=1 << 30, stream=None)),
    "gdr_lru_step": (lru, dict(slots=None, x=16, r=16, i=16, lam=16, h=16, y=16, stream=None)),
    "gdr_layernorm_forward": (ln, dict(x=16, residual=16, w=16, b=16, y=16, r=16, stream=None)),
    "gdr_layernorm_backward": (ln, dict(dy=16, r=16, w=16, dr=16, dx=16, dw=16, db=16, ws=256, nbytes=1 << 30,
                                        stream=None)),
    "gdr_gated_norm_forward": (gn, dict(x=16, z=16, w=16, y=16, stream=None)),
    "gdr_gated_norm_backward": (gn, dict(dy=16, x=16, z=16, w=16, dx=16, dz=16, dw=16, ws=256, nbytes=1 << 30,
                                         stream=None)),
}
REQUIRED = {
    "gdr_lru_forward": ["x", "r", "y"], "gdr_lru_backward": ["x", "r", "dy", "dx", "dr", "di", "dlam"],
    "gdr_lru_step": ["x", "r", "h", "y"], "gdr_layernorm_forward": ["x", "w"],
    "gdr_layernorm_backward": ["dy", "r", "w", "dx", "dw", "db"], "gdr_gated_norm_forward": ["x", "z", "w", "y"],
    "gdr_gated_norm_backward": ["dy", "x", "z", "w", "dx", "dz", "dw"],
}


@pytest.mark.parametrize("name", CALLS)
def test_null_problem(lib, name):
    assert call(name, None, CALLS[name][1].values()) == NULL


@pytest.mark.parametrize("name,ptr", [(n, p) for n, ps in REQUIRED.items() for p in ps])
def test_null_required_pointer(lib, name, ptr):
    make, ptrs = CALLS[name]
    assert call(name, make(), (ptrs | {ptr: None}).values()) == NULL


@pytest.mark.parametrize("name,ptr", [(n, p) for n, (_, ps) in CALLS.items() for p in ps
                                      if p not in ("stream", "nbytes", "ws")])
def test_misaligned_pointer(lib, name, ptr):
    make, ptrs = CALLS[name]
    assert call(name, make(), (ptrs | {ptr: 17}).values()) == ALIGN


@pytest.mark.parametrize("name", [n for n, (_, p) in CALLS.items() if "ws" in p])
def test_workspace(lib, name):
    make, ptrs = CALLS[name]
    p, more = make(), {"gdr_lru_forward": [0], "gdr_lru_backward": [0, 1]}.get(name, [])
    need = getattr(lib, name + "_workspace_bytes")(ctypes.byref(p), *more)
    assert need > 0
    assert call(name, p, (ptrs | dict(ws=None)).values()) == WORKSPACE
    assert call(name, p, (ptrs | dict(nbytes=need - 1)).values()) == WORKSPACE
    assert call(name, p, (ptrs | dict(ws=128)).values()) == ALIGN
    assert getattr(lib, name + "_workspace_bytes")(None, *more) == 0
    p.io_dtype = 7
    assert getattr(lib, name + "_workspace_bytes")(ctypes.byref(p), *more) == 0


def test_without_kept_states_the_gradient_needs_more(lib):
    p = ctypes.byref(lru())
    assert lib.gdr_lru_backward_workspace_bytes(p, 0, 0) > lib.gdr_lru_backward_workspace_bytes(p, 0, 1)
    assert lib.gdr_lru_kept_bytes(p, 0) == 2 * 4 * 64 * 4          # two sequences of four tiles
    assert lib.gdr_lru_kept_bytes(p, 1) == (1000 // 128 + 2) * 64 * 4
    assert lib.gdr_lru_kept_bytes(None, 0) == 0


@pytest.mark.parametrize("name", CALLS)
def test_bad_dtype(lib, name):
    make, ptrs = CALLS[name]
    assert call(name, make(io_dtype=3), ptrs.values()) == DTYPE


@pytest.mark.parametrize("name,kw,status", [
    ("gdr_lru_forward", dict(n=0), SHAPE), ("gdr_lru_forward", dict(T=0), SHAPE), ("gdr_lru_forward", dict(D=0), SHAPE),
    ("gdr_lru_forward", dict(D=(1 << 20) + 1), SHAPE), ("gdr_lru_forward", dict(x_ld=63), SHAPE),
    ("gdr_lru_forward", dict(r_ld=1), SHAPE), ("gdr_lru_forward", dict(i_ld=-64), SHAPE),
    ("gdr_lru_forward", dict(c=0.0), ARG), ("gdr_lru_forward", dict(c=-1.0), ARG),
    ("gdr_lru_forward", dict(c=float("nan")), ARG), ("gdr_lru_forward", dict(c=float("inf")), ARG),
    ("gdr_lru_forward", dict(n=1 << 30, T=1), SHAPE), ("gdr_lru_forward", dict(n=1 << 20, T=1 << 12), SHAPE),
    ("gdr_lru_forward", dict(n=1 << 20, T=1, D=1 << 20), SHAPE),        # more blocks than a grid takes
    ("gdr_lru_backward", dict(T=-4), SHAPE), ("gdr_lru_backward", dict(c=float("nan")), ARG),
    ("gdr_lru_step", dict(n=5), SHAPE), ("gdr_lru_step", dict(pool=0), SHAPE), ("gdr_lru_step", dict(pool=1 << 30), SHAPE),
    ("gdr_layernorm_forward", dict(rows=-1), SHAPE), ("gdr_layernorm_forward", dict(rows=1 << 30), SHAPE),
    ("gdr_layernorm_forward", dict(D=0), SHAPE), ("gdr_layernorm_forward", dict(D=32769), SHAPE),
    ("gdr_layernorm_forward", dict(x_ld=63), SHAPE), ("gdr_layernorm_forward", dict(res_ld=63), SHAPE),
    ("gdr_layernorm_forward", dict(eps=float("nan")), ARG), ("gdr_layernorm_forward", dict(eps=float("inf")), ARG),
    ("gdr_layernorm_backward", dict(eps=-1e-6), ARG),
    ("gdr_gated_norm_forward", dict(tokens=-1), SHAPE), ("gdr_gated_norm_forward", dict(H=0), SHAPE),
    ("gdr_gated_norm_forward", dict(V=0), SHAPE), ("gdr_gated_norm_forward", dict(V=8193), SHAPE),
    ("gdr_gated_norm_forward", dict(tokens=1 << 29), SHAPE), ("gdr_gated_norm_forward", dict(x_ld=127), SHAPE),
    ("gdr_gated_norm_forward", dict(z_ld=127), SHAPE), ("gdr_gated_norm_forward", dict(gate=2), ARG),
    ("gdr_gated_norm_forward", dict(per_head=-1), ARG), ("gdr_gated_norm_forward", dict(eps=float("nan")), ARG),
    ("gdr_gated_norm_backward", dict(eps=float("inf")), ARG),
])
def test_bad_problem(lib, name, kw, status):
    make, ptrs = CALLS[name]
    assert call(name, make(**kw), ptrs.values()) == status


def test_packed_tokens_beyond_31_bit_tiles(lib):
    _, ptrs = CALLS["gdr_lru_forward"]
    assert call("gdr_lru_forward", lru(n=1, total=1 << 30), (ptrs | dict(cu=16)).values()) == SHAPE


def test_nothing_to_write_and_nothing_to_do(lib):
    _, ptrs = CALLS["gdr_layernorm_forward"]
    assert call("gdr_layernorm_forward", ln(), (ptrs | dict(y=None, r=None)).values()) == NULL
    assert call("gdr_layernorm_forward", ln(rows=0), [None] * 7) == 0
    assert call("gdr_gated_norm_forward", gn(tokens=0), [None] * 5) == 0


def test_the_binding_refuses_host_tensors(lib):
    import torch
    from chunked_gated_delta_prepare_gb300 import layer
    x, w = torch.zeros(2, 64), torch.zeros(64)
    for f in (lambda: layer.lru_forward(x[None], x[None]), lambda: layer.lru_backward(x[None], x[None], None, None, x[None]),
              lambda: layer.lru_step(x, x, None, None, x), lambda: layer.layernorm_forward(x, w),
              lambda: layer.layernorm_backward(x, x, w), lambda: layer.gated_norm_forward(x, x, w),
              lambda: layer.gated_norm_backward(x, x, x, w), lambda: layer.lru_forward(None, x),
              lambda: layer.layernorm_forward(None, w), lambda: layer.gated_norm_forward([1.0], x, w),
              lambda: layer.lru_forward(x[None], x[None], stream=1234)):
        with pytest.raises(ValueError):
            f()
