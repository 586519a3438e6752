"""The example model's layer of the gated linear recurrence: decoding against the whole prompt, and its gradients."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    import recurrent_model
    return recurrent_model


@pytest.mark.parametrize("kinds", [("lru",), ("lru", "delta", "ssm", "lru")])
def test_decoding_goes_on_from_packed_prompts(example, kinds):
    # as for the other kinds: bf16 activations between two orders of the same sums, a few percent of the largest logit
    gap, top = example.decode_gap(example.Model(kinds))
    assert gap <= 0.05 * top


def plain(e, one, x, residual):
    """The layer's training pass by its formulas, in the inputs' type."""
    r = x + residual
    p = F.layer_norm(r, (e.DIM,), one["norm"], one["norm_bias"], 1e-5) @ one["inp"].t()
    c, gate, inlet, z = p.split(e.INNER, -1)
    c = F.conv1d(F.pad(c.transpose(1, 2), (e.TAPS - 1, 0)), one["taps"].unsqueeze(1), one["bias"], groups=e.INNER)
    c = F.silu(c).transpose(1, 2)
    decay = -8.0 * F.softplus(one["lam"]) * torch.sigmoid(gate)
    inflow = torch.sqrt(-torch.expm1(2 * decay)) * torch.sigmoid(inlet) * c
    h, hs = torch.zeros_like(c[:, 0]), []
    for t in range(c.shape[1]):
        h = torch.exp(decay[:, t]) * h + inflow[:, t]
        hs.append(h)
    o = torch.stack(hs, 1).unflatten(-1, (-1, e.HEAD))
    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * one["gain"] * F.silu(z.unflatten(-1, (-1, e.HEAD)))
    return o.flatten(2) @ one["out"].t(), r


def test_gradients_of_the_layer(example):
    """Every parameter's and input's gradient against the formulas' in 64 bits."""
    torch.manual_seed(0)
    one = example.Layer("lru", torch.Generator().manual_seed(3))
    names = [k for k, v in vars(one).items() if isinstance(v, torch.Tensor)]
    x, res, do, dr = (torch.randn(2, 150, example.DIM, device="cuda").to(example.IO) for _ in range(4))
    leaves = [x, res] + [getattr(one, k) for k in names]
    for t in leaves:
        t.requires_grad_(True)
    out, r = one.train(x, res)
    got = torch.autograd.grad((out, r), leaves, (do, dr))
    wide = [t.detach().double().requires_grad_(True) for t in leaves]
    ref_out, ref_r = plain(example, dict(zip(names, wide[2:])), *wide[:2])
    want = torch.autograd.grad((ref_out, ref_r), wide, (do.double(), dr.double()))
    # A dozen tensors on the way forth and a dozen on the way back are rounded to bf16, each by at most 2^-8 of its
    # values; norms, gates and the recurrence's decay pass a relative error on at about its size: 24 * 2^-8 = 0.094.
    for name, a, b in zip(["x", "residual"] + names, got, want):
        gap = float((a.double() - b).norm() / b.norm())
        assert gap <= 0.094, (name, gap)
    out, ref_out = out.detach().double(), ref_out.detach()
    assert float((out - ref_out).norm() / ref_out.norm()) <= 0.094


@pytest.mark.parametrize("kinds", [("lru",), ("delta", "lru", "ssm")])
def test_model_trains(example, kinds):
    model = example.Model(kinds)
    losses = example.train(model, steps=3)
    assert torch.isfinite(torch.tensor(losses)).all()
    assert all(torch.isfinite(p).all() for p in model.parameters())


def test_main_runs(example, capsys):
    example.main()
    assert "training" in capsys.readouterr().out
