"""The gated delta rule's single-token step against the recurrence in 64 bits, and against the prompt's forward.

Tolerances.  A state element is three fp32 operations after sums over K = 128 terms: it is held to 1e-5 of the largest
size its column's terms reach, o (before its rounding to the io type) likewise.  The forward works in its io type's
products, so a step after a prompt is compared with fp32 io, at 1e-4 of the output's largest value.
"""
import math

import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, forward, layer
from chunked_gated_delta_prepare_gb300.inputs import make_inputs

pytestmark = pytest.mark.gpu
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(B, H, HV, K, V, per_k, io, pool, seed=0):
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    q, k = (torch.nn.functional.normalize(randn(B, H, K), dim=-1).to(io).cuda() for _ in range(2))
    v, beta = randn(B, HV, V).to(io).cuda(), torch.rand(B, HV, generator=gen).to(io).cuda()
    g = -torch.rand(B, HV, K, generator=gen).cuda() if per_k else -torch.rand(B, HV, generator=gen).cuda()
    h = randn(pool, HV, K, V).cuda()
    return q, k, v, g, beta, h


def reference(q, k, v, g, beta, h, scale):
    per = v.shape[1] // q.shape[1]
    q, k = (t.double().repeat_interleave(per, 1) for t in (q, k))
    decay = torch.exp(g.double())
    S = h.double() * (decay[..., None] if g.dim() == 3 else decay[..., None, None])
    delta = beta.double()[..., None] * (v.double() - torch.einsum("bhkv,bhk->bhv", S, k))
    size = S.abs().amax(-2) * math.sqrt(k.shape[-1]) + delta.abs()
    S = S + k[..., :, None] * delta[..., None, :]
    return S, scale * torch.einsum("bhkv,bhk->bhv", S, q), size


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("per_k", [False, True])
@pytest.mark.parametrize("B,H,HV,K,V", [(1, 1, 1, 64, 64), (3, 2, 6, 128, 64), (2, 3, 3, 64, 128), (70, 2, 4, 128, 128)])
def test_step(B, H, HV, K, V, per_k, io):
    pool = B + 3
    q, k, v, g, beta, h = make(B, H, HV, K, V, per_k, io, pool)
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32).cuda()
    live = torch.ones(B, dtype=torch.bool)
    if B > 1:
        slots[1], live[1] = -1, False
        q[1], v[1], g[1] = float("nan"), float("inf"), float("inf")
    if B > 2:
        slots[2], live[2] = pool + 7, False
    before = h.clone()
    o = layer.delta_step(q, k, v, g, beta, h, slots=slots)
    at = slots[live.cuda()].long()
    S, want, size = reference(*(t[live.cuda()] for t in (q, k, v, g, beta)), before[at], 1 / math.sqrt(K))
    assert bool(((h[at].double() - S).abs() <= 1e-5 * size[..., None, :]).all())
    assert bool(((o[live.cuda()].double() - want).abs() <= 1e-5 * size + HALF_ULP[io] * want.abs() + 2.0 ** -24).all())
    assert not o[~live.cuda()].any()
    before[at] = h[at]
    assert torch.equal(before, h)              # no other state moved


def test_slices_scale_and_no_slots():
    B, H, HV, K, V = 5, 2, 4, 64, 128
    q, k, v, g, beta, h = make(B, H, HV, K, V, False, torch.bfloat16, 6)
    row = torch.cat([torch.zeros(B, 3, device="cuda", dtype=torch.bfloat16), q.flatten(1), k.flatten(1), v.flatten(1)], 1)
    qs, ks, vs = row[:, 3:].split([H * K, H * K, HV * V], 1)
    h2 = h.clone()
    o = layer.delta_step(q, k, v, g, beta, h, scale=0.5)
    o2 = layer.delta_step(qs.unflatten(1, (H, K)), ks.unflatten(1, (H, K)), vs.unflatten(1, (HV, V)), g, beta, h2,
                          scale=0.5)
    assert torch.equal(o, o2) and torch.equal(h, h2)
    S, want, size = reference(q, k, v, g, beta, make(B, H, HV, K, V, False, torch.bfloat16, 6)[-1][:B], 0.5)
    assert bool(((o.double() - want).abs() <= 1e-5 * size + 2.0 ** -8 * want.abs()).all())


@pytest.mark.parametrize("per_k", [False, True])
def test_steps_go_on_from_a_prompt(per_k):
    x = make_inputs(2, 40, 3, 64, 64, per_k_gate=per_k, io_dtype=torch.float32, seed=3)
    q, k, v, g, beta = (t.cuda() for t in (x.q, x.k, x.v, x.g, x.beta))
    whole, last = forward(q, k, v, g, beta, chunk=32)
    _, h = forward(*(t[:, :33].contiguous() for t in (q, k, v, g, beta)), chunk=32)
    for t in range(33, 40):
        o = layer.delta_step(*(y[:, t].contiguous() for y in (q, k, v, g, beta)), h)
        assert float((o - whole[:, t]).abs().max()) <= 1e-4 * float(whole.abs().max())
    assert float((h - last).abs().max()) <= 1e-4 * float(last.abs().max())


def test_another_stream():
    side = torch.cuda.Stream()
    q, k, v, g, beta, h = make(64, 8, 8, 128, 128, False, torch.bfloat16, 64)
    h2 = h.clone()
    side.wait_stream(torch.cuda.current_stream())
    o = layer.delta_step(q, k, v, g, beta, h, stream=side)
    side.synchronize()
    assert torch.equal(o, layer.delta_step(q, k, v, g, beta, h2)) and torch.equal(h, h2)


def test_refusals():
    q, k, v, g, beta, h = make(2, 2, 4, 64, 64, False, torch.bfloat16, 3)
    for args in ((q, k[:, :1], v, g, beta, h), (q, k, v, g[:1], beta, h), (q, k, v, g.double(), beta, h),
                 (q, k, v, g, beta.float(), h), (q, k, v, g, beta, h.double()), (q, k, v.float(), g, beta, h),
                 (q, k, v, g, beta, h.transpose(2, 3)), (q, k, v, g, beta, h[:, :2]), (q.cpu(), k, v, g, beta, h)):
        with pytest.raises(ValueError):
            layer.delta_step(*args)
    with pytest.raises(ValueError):
        layer.delta_step(q, k, v, g, beta, h, slots=torch.zeros(2, device="cuda"))
    for args, kw, status in (((q, k, v, g, beta, h[:1].contiguous()), {}, 2),                 # two rows, one state
                             ((q, k, v, g, beta, h), dict(scale=float("nan")), 9),
                             (make(1, 1, 1, 32, 64, False, torch.float32, 1), {}, 2),
                             (make(1, 2, 3, 64, 64, False, torch.float32, 1), {}, 2)):
        with pytest.raises(GdrError) as e:
            layer.delta_step(*args, **kw)
        assert e.value.status == status
