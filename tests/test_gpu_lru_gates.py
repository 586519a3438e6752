"""The gated linear recurrence with gates far open and far shut: small factors keep their digits.

Tolerances are those of test_gpu_lru.py and test_gpu_lru_backward.py, of the terms' own sizes and with nothing beside them:
each of a, 1 - a, sigmoid(r), 1 - sigmoid(r), g, 1 - g is a product of e^-r or e^-i (whose exponent, up to 29, is rounded to
2^-20 twice: 1.4e-6) with a reciprocal or a root (2^-22).
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import layer
from lru_reference import scan_backward
from test_gpu_lru import FORMS, make, part
from test_gpu_lru_backward import TOL as GRAD_TOL, randn

pytestmark = pytest.mark.gpu
INF = float("inf")


def wide_gates(s, lo=-20.0, hi=20.0, seed=5):
    gen = torch.Generator().manual_seed(seed)
    for key in ("r", "i"):
        if s[key] is not None:
            s[key] = (lo + (hi - lo) * torch.rand(*s[key].shape, generator=gen)).to(s[key].dtype).cuda()
    return s


def relative(s, dy, got, c=8.0):
    for b in range(dy.shape[0]):
        want = scan_backward(**part(s, b), dy=dy[b], h0=s["h0"][b], c=c)
        for name in ("dx", "dr", "di", "dh0"):
            have = getattr(got, name)
            if have is not None:
                v, size = want[name]
                err = (have[b].double() - v).abs()
                assert bool((err <= GRAD_TOL * size).all()), (name, float((err / size.clamp_min(1e-300)).max()))


@pytest.mark.parametrize("c", [8.0, 1.5])
@pytest.mark.parametrize("form,gate", [f for f in FORMS if f[0] == "rate"])
@pytest.mark.parametrize("T,D", [(160, 72), (9, 5)])
def test_gradients_of_open_and_shut_gates(T, D, form, gate, c):
    s = wide_gates(make((2, T), D, torch.float32, form, gate))
    dy = 1e4 * randn(2, T, D, seed=1)
    relative(s, dy, layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], c=c), c)


@pytest.mark.parametrize("T,D", [(160, 72), (9, 5)])
def test_gradient_of_an_open_input_gate_without_rates(T, D):
    """di holds 1 - g, which is 2e-9 at i = 20."""
    s = wide_gates(make((2, T), D, torch.float32, "direct"), 4.0)
    s["r"] = torch.randn(2, T, D, generator=torch.Generator().manual_seed(3)).cuda()
    dy = 1e4 * randn(2, T, D, seed=1)
    relative(s, dy, layer.lru_backward(s["x"], s["r"], s["i"], None, dy, s["h0"]))


@pytest.mark.parametrize("form,gate", FORMS)
def test_gates_at_infinity_have_no_gradient(form, gate):
    s = make((1, 140), 70, torch.float32, form, gate)
    s["r"][0, ::7], s["r"][0, 3::7] = INF, -INF
    if gate:
        s["i"][0, 1::5], s["i"][0, 2::5] = INF, -INF
    dy = 1e4 * randn(1, 140, 70, seed=1)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"])
    assert all(g is None or bool(g.isfinite().all()) for g in got)
    assert not got.dr[s["r"].isinf()].any()
    if gate:
        assert not got.di[s["i"].isinf()].any() and not got.dx[s["i"] == -INF].any()
