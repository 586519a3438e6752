"""The gated norm's gradient with eps = 0, where a row that is not there must add nothing to the weights' sums.

Tolerances: those of test_gpu_gated_norm.py.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import layer
from test_gpu_gated_norm import HALF_ULP, gate_of, make

pytestmark = pytest.mark.gpu


# rows that are no multiple of a block's, and tokens that are no multiple of what a wave of places takes
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("tokens,H,V", [(3, 1, 64), (10001, 1, 64), (5, 3, 128), (2000, 3, 512), (700, 1, 4096)])
def test_gradient_with_eps_zero(tokens, H, V, per_head, io):
    x, z, w = make(tokens, H, V, io, per_head)
    dy = torch.randn(tokens, H, V, generator=torch.Generator().manual_seed(1)).to(io).cuda()
    dx, dz, dw = layer.gated_norm_backward(dy, x, z, w, eps=0.0)
    f, _, _ = gate_of(z, "silu")
    xd, wd, g = x.double(), w.double(), dy.double()
    rstd = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True))
    n, dn = xd * rstd, g * wd * f
    dot = (dn * n).mean(-1, keepdim=True)
    want = rstd * (dn - n * dot)
    size = rstd * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True))
    assert bool(((dx.double() - want).abs() <= 1e-5 * size + HALF_ULP[io] * want.abs() + 2.0 ** -24).all())
    assert bool(dz.isfinite().all())
    over = (0,) if per_head else (0, 1)
    err, terms = (dw.double() - (g * n * f).sum(over)).abs(), (g * n * f).abs().sum(over)
    assert bool((err <= 2.6e-5 * terms).all()), float((err / terms).max())
