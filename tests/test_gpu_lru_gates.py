"""The gated linear recurrence with gates far open and far shut: small factors keep their digits.

Tolerances are those of test_gpu_lru.py and test_gpu_lru_backward.py, of the terms' own sizes and with nothing beside them:
each of a, 1 - a, sigmoid(r), 1 - sigmoid(r), g, 1 - g is a product of e^-r or e^-i (whose exponent, up to 29, is rounded to
2^-20 twice: 1.4e-6) with a reciprocal or a root (2^-22).
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import layer
from lru_reference import scan_backward
from test_gpu_lru import FORMS, TOL, make, part
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


# ---------------------------------------------------------------- a shut forget gate

@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T,D", [(160, 72), (9, 5)])
def test_gradients_of_a_shut_forget_gate(T, D, gate):
    """Without rates dr holds a = sigmoid(r), 2e-9 at r = -20."""
    s = wide_gates(make((2, T), D, torch.float32, "direct", gate))
    dy = 1e4 * randn(2, T, D, seed=1)
    relative(s, dy, layer.lru_backward(s["x"], s["r"], s["i"], None, dy, s["h0"]))
    s["r"] = s["r"].abs().neg()
    relative(s, dy, layer.lru_backward(s["x"], s["r"], s["i"], None, dy, s["h0"]))


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [True, False])
def test_what_a_shut_forget_gate_leaves(gate, io):
    """Nothing flows in, so a state is the product of its decays: 3 of them at a time, from states of 1e18."""
    D = 2000
    s = wide_gates(make((1, 3), D, io, "direct", gate), -20.0, -5.0)
    s["x"].zero_()
    s["h0"] = 1e18 * s["h0"]
    y, h, _ = layer.lru_forward(**s)
    pool = s["h0"].clone()
    want, ulp = s["h0"][0].double(), {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}[io]
    for t in range(3):
        want = want * torch.sigmoid(s["r"][0, t].double())
        row = (s["x"][0, t][None], s["r"][0, t][None], None if s["i"] is None else s["i"][0, t][None])
        step = layer.lru_step(*row, None, pool)
        for got in (y[0, t], step[0]):
            assert bool(((got.double() - want).abs() <= (TOL + ulp) * want.abs()).all())
    for got in (h[0], pool[0]):
        assert bool(((got.double() - want).abs() <= TOL * want.abs()).all())


@pytest.mark.parametrize("gate", [True, False])
def test_what_flows_in_behind_a_shut_forget_gate(gate):
    """All of the input, up to where e^-r is infinite."""
    shut = torch.tensor([-20.0, -27.5, -60.0, -86.5, -87.4, -87.5, -87.7, -88.0, -88.5, -100.0, -INF], device="cuda")
    s = make((1, len(shut)), 6, torch.float32, "direct", gate)
    s["r"] = shut[None, :, None].expand_as(s["x"]).contiguous()
    want = s["x"].double() * (torch.sigmoid(s["i"].double()) if gate else 1.0)
    y, _, _ = layer.lru_forward(**s)
    pool, dy = s["h0"].clone(), randn(1, len(shut), 6, seed=1)
    d = layer.lru_backward(s["x"], s["r"], s["i"], None, dy, s["h0"])
    size = want.abs() + torch.cat([s["h0"].double()[None], want[:, :-1].abs()], 1).abs() * torch.sigmoid(s["r"].double())
    assert bool(((y.double() - want).abs() <= TOL * size + size - want.abs()).all())
    e = dy.double() * (torch.sigmoid(s["i"].double()) if gate else 1.0)
    after = torch.cat([dy[:, 1:], torch.zeros_like(dy[:, :1])], 1).double().abs() * 2.1e-9       # what a later token sends back
    assert bool(((d.dx.double() - e).abs() <= GRAD_TOL * e.abs() + after).all())
    for t in range(len(shut)):
        step = layer.lru_step(s["x"][0, t][None], s["r"][0, t][None], None if s["i"] is None else s["i"][0, t][None], None, pool)
        assert bool(((step.double() - want[0, t]).abs() <= TOL * size[0, t] + size[0, t] - want[0, t].abs()).all())
