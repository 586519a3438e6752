"""The gated linear recurrence: a token's bits follow from its own channel's numbers; rates on both sides of 1/4.

Tolerances are those of test_gpu_lru.py and test_gpu_lru_backward.py.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import layer
from test_gpu_lru import FORMS, TYPES, check, make
from test_gpu_lru_backward import compare, randn

pytestmark = pytest.mark.gpu
INF = float("inf")


def equal(a, b, at):
    return all(u is None or torch.equal(u[at], v[at]) for u, v in zip(a, b))


@pytest.mark.parametrize("D", [70, 71, 72])
@pytest.mark.parametrize("value", [float("nan"), -INF, -100.0, -40.0, INF])
@pytest.mark.parametrize("form,gate", FORMS)
def test_a_gate_is_its_own_channels_and_tokens(form, gate, value, D):
    """The other channels, and what does not follow from the gate in its own, have the same bits whatever it is."""
    s = make((1, 300), D, torch.float32, form, gate)
    dy = randn(1, 300, D, seed=1)

    def run():
        y, _, _ = layer.lru_forward(**s)
        d = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"])
        return (y, d.dx, d.dr, d.di)

    clean, others = run(), torch.arange(D, device="cuda") != 11
    for key in ("r", "i") if gate else ("r",):
        keep = s[key].clone()
        s[key][0, 140, 11] = value
        got = run()
        s[key] = keep
        assert equal(got, clean, (slice(None), slice(None), others)), key
        assert torch.equal(got[0][0, :140, 11], clean[0][0, :140, 11]), key
        if key == "i":                               # e does not follow from the input's gate
            assert equal(got, clean, (0, slice(0, 140), 11)) and torch.equal(got[1][0, 141:, 11], clean[1][0, 141:, 11])


def test_a_rate_is_its_own_channels():
    s = make((1, 300), 70, torch.float32)
    dy = randn(1, 300, 70, seed=1)

    def run():
        y, _, kept = layer.lru_forward(**s, want_kept=True)
        d = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], kept=kept)
        return (y, d.dx, d.dr, d.di)

    clean, others = run(), torch.arange(70, device="cuda") % 8 != 3
    s["lam"][3::8] = 0.5                              # k = 7.8
    assert equal(run(), clean, (slice(None), slice(None), others))


def test_channels_cut_anywhere():
    """A tensor's channels from the second on, by themselves: pairs of other channels, the same bits."""
    s = make((1, 300), 67, torch.float32)
    s["lam"][::3] = 0.0
    dy = randn(1, 300, 67, seed=1)
    cut = {k: (None if v is None else v[..., 1:].contiguous()) for k, v in s.items()}
    whole, less = (layer.lru_forward(**v)[0] for v in (s, cut))
    assert torch.equal(whole[..., 1:], less)
    a = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"])
    b = layer.lru_backward(cut["x"], cut["r"], cut["i"], cut["lam"], dy[..., 1:].contiguous(), cut["h0"])
    for name in ("dx", "dr", "di"):
        assert torch.equal(getattr(a, name)[..., 1:], getattr(b, name)), name


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form,gate", FORMS)
def test_channels_by_either_way_into_shared_memory(form, gate, io):
    """Rows on 16-byte boundaries and rows that start anywhere take other kernels: the same bits."""
    s = make((3, 300), 72, io, form, gate)
    if form == "rate":
        s["lam"][::5] = 0.0
    dy = randn(3, 300, 72, io=io, seed=1)
    cut = {k: (None if v is None else v[..., :67].contiguous()) for k, v in s.items()}
    (y, h, kept), (y1, h1, kept1) = (layer.lru_forward(**v, want_kept=True) for v in (s, cut))
    assert torch.equal(y[..., :67], y1) and torch.equal(h[:, :67], h1) and torch.equal(kept[:, :67], kept1)
    a = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], kept=kept)
    b = layer.lru_backward(cut["x"], cut["r"], cut["i"], cut["lam"], dy[..., :67].contiguous(), cut["h0"], kept=kept1)
    for name in ("dx", "dr", "di", "dh0", "dlam"):
        u, v = getattr(a, name), getattr(b, name)
        assert u is None or torch.equal(u[..., :67], v), name


# ---------------------------------------------------------------- rates on both sides of 1/4

@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("most", [0.84, 5.0])
def test_rates_up_to(most, gate, io):
    """Whole tiles, and a part of one, of channels whose k = c softplus(lam) goes from 1/20 to `most`."""
    D = 200
    s = make((2, 300), D, io, "rate", gate)
    k = torch.linspace(0.05, most, D)[torch.randperm(D, generator=torch.Generator().manual_seed(2))]
    s["lam"] = torch.log(torch.expm1(k / 8)).cuda()
    dy, dh = randn(2, 300, D, io=io, seed=1), randn(2, D, seed=2)
    y, h, kept = layer.lru_forward(**s, want_kept=True)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], dh, kept)
    for b in range(2):
        check(s, b, b, y, h, io)
    compare(s, range(2), dy, dh, got, io)
