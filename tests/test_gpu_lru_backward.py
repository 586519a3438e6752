"""The gradient of the gated linear recurrence against the reverse recurrence in 64 bits and against differences.

Tolerances.  Every term is a product of a state, a state's gradient and a few inputs; both chains carry the forward's
error of 2e-5 of their terms (test_gpu_lru.py), so gradients are held to 5e-5 of the sum of their terms' sizes, and
16-bit ones to half a unit in the last place on top.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, layer
from lru_reference import scan, scan_backward
from test_gpu_lru import FORMS, HALF_ULP, LENGTHS, SHAPES, TYPES, bounds, make, part

pytestmark = pytest.mark.gpu
TOL = 5e-5


def randn(*shape, io=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(io).cuda()


def compare(s, rows_of, dy, dh, got, io, c=8.0, floor=1e-30):
    """rows_of: the leading index of each sequence's tokens; floor: what dlam may be off by beside its terms."""
    total = None
    for i, rows in enumerate(rows_of):
        want = scan_backward(**part(s, rows), dy=dy[rows], h0=None if s["h0"] is None else s["h0"][i],
                             dh_final=None if dh is None else dh[i], c=c)
        for name in ("dx", "dr", "di", "dh0"):
            have = getattr(got, name)
            if have is None:
                continue
            v, size = want[name]
            have = have[i] if name == "dh0" else have[rows]
            ulp = 0.0 if name == "dh0" else HALF_ULP[io]
            err = (have.double() - v).abs()
            tiny = 1e-30 if name == "dh0" else 2.0 ** -24
            assert bool((err <= TOL * size + ulp * v.abs() + tiny).all()), (name, i, float(err.max()))
        if "dlam" in want:
            total = want["dlam"] if total is None else [a + b for a, b in zip(total, want["dlam"])]
    if total is not None:
        err = (got.dlam.double() - total[0]).abs()
        assert bool((err <= TOL * total[1] + floor).all()), float((err / total[1].clamp_min(1e-30)).max())


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form,gate", FORMS)
@pytest.mark.parametrize("B,T,D,pad", SHAPES)
def test_batches(B, T, D, pad, form, gate, io):
    s = make((B, T), D, io, form, gate, pad=pad, h0=T % 2 == 1)
    dy = randn(B, T, D, io=io, seed=1)
    dh = randn(B, D, seed=2) if T % 3 else None
    _, _, kept = layer.lru_forward(**s, want_kept=True)
    args = (s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], dh)
    got = layer.lru_backward(*args, kept)
    assert (got.di is not None) == gate and (got.dlam is not None) == (form == "rate")
    assert (got.dh0 is not None) == (s["h0"] is not None)
    compare(s, range(B), dy, dh, got, io)
    for again in (layer.lru_backward(*args, kept), layer.lru_backward(*args)):     # the states formed again: the same bits
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,form,gate", [(40, "rate", True), (264, "direct", True), (65, "direct", False), (7, "rate", False)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, D, form, gate, io):
    s = make((sum(lens),), D, io, form, gate, n=len(lens))
    cu, rows = bounds(lens)
    dy, dh = randn(sum(lens), D, io=io, seed=1), randn(len(lens), D, seed=2)
    _, _, kept = layer.lru_forward(**s, cu_seqlens=cu, want_kept=True)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], dh, kept, cu_seqlens=cu)
    compare(s, rows, dy, dh, got, io)
    again = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], dh, cu_seqlens=cu)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


def test_a_sequence_does_not_see_its_neighbours():
    cu, rows = bounds([100, 190, 300])
    s = make((590,), 72, torch.float32, n=3)
    dy = randn(590, 72, seed=1)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], cu_seqlens=cu)
    bad = {k: (v if k == "lam" else v.clone()) for k, v in s.items()}
    for t in (bad["x"], bad["r"], bad["i"], dy):
        t[:100], t[290:] = float("nan"), float("inf")
    bad["h0"][0] = float("nan")
    out = layer.lru_backward(bad["x"], bad["r"], bad["i"], bad["lam"], dy, bad["h0"], cu_seqlens=cu)
    for name in ("dx", "dr", "di"):
        assert torch.equal(getattr(got, name)[rows[1]], getattr(out, name)[rows[1]]), name
    assert torch.equal(got.dh0[1], out.dh0[1])


@pytest.mark.parametrize("form,gate", FORMS)
def test_against_differences(form, gate):
    s = make((1, 6), 4, torch.float32, form, gate)
    dy, dh = randn(1, 6, 4, seed=1), randn(1, 4, seed=2)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], dh)
    names = dict(x="dx", r="dr", i="di", lam="dlam", h0="dh0")

    def loss(v):
        hs, _ = scan(v["x"][0], v["r"][0], None if v["i"] is None else v["i"][0], v["lam"], v["h0"][0])
        return float((hs[1:] * dy[0].double()).sum() + (hs[-1] * dh[0].double()).sum())

    base, h = {k: None if v is None else v.double().contiguous() for k, v in s.items()}, 1e-5
    for key, name in names.items():
        if base[key] is None:
            continue
        grad = getattr(got, name).reshape(-1)
        for j in range(0, base[key].numel(), 3):
            hi, lo = ({k: None if v is None else v.clone() for k, v in base.items()} for _ in range(2))
            hi[key].view(-1)[j] += h
            lo[key].view(-1)[j] -= h
            assert float(grad[j]) == pytest.approx((loss(hi) - loss(lo)) / (2 * h), rel=1e-4, abs=1e-4), (key, j)


def test_gates_at_their_ends_have_finite_gradients():
    """sqrt(1 - a^2) has an infinite slope where a = 1; what multiplies it there is zero."""
    s = make((1, 40), 6, torch.float32)
    s["lam"] = torch.tensor([-200.0, -100.0, -30.0, 20.0, 200.0, 0.0], device="cuda")
    s["r"][0, 3], s["r"][0, 7], s["i"][0, 9], s["i"][0, 12] = -float("inf"), -200.0, -float("inf"), 100.0
    s["r"][0, 5], s["r"][0, 30] = float("inf"), 90.0
    dy = randn(1, 40, 6, seed=1)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"])
    assert all(bool(g.isfinite().all()) for g in got)
    # softplus(-100) = 3.7e-44 lies below fp32's normal numbers, whose step there is 1.4e-45: it is off by up to half a step,
    # 1.9 %, and dlam, which goes with its root, by 1 % of its terms' 7.6e-20
    compare(s, [0], dy, None, got, torch.float32, floor=7.6e-22)
    s = make((1, 40), 6, torch.float32, "direct")
    s["r"][0, 3], s["r"][0, 7], s["r"][0, 20] = -float("inf"), float("inf"), 200.0
    got = layer.lru_backward(s["x"], s["r"], s["i"], None, dy, s["h0"])
    assert all(g is None or bool(g.isfinite().all()) for g in got)
    compare(s, [0], dy, None, got, torch.float32)


def test_strided_gradients_are_copied():
    s = make((2, 150), 24, torch.bfloat16)
    dy = randn(150, 2, 24, io=torch.bfloat16, seed=1).transpose(0, 1)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"])
    want = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy.contiguous(), s["h0"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_bits_again_and_on_another_stream():
    s = make((5000,), 600, torch.bfloat16, n=3)
    cu, _ = bounds([4000, 0, 1000])
    dy = randn(5000, 600, io=torch.bfloat16, seed=1)
    args = (s["x"], s["r"], s["i"], s["lam"], dy, s["h0"])
    want = layer.lru_backward(*args, cu_seqlens=cu)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, layer.lru_backward(*args, cu_seqlens=cu)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer.lru_backward(*args, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    s = make((2, 5), 8, torch.bfloat16)
    dy = randn(2, 5, 8, io=torch.bfloat16)
    args = dict(x=s["x"], r=s["r"], i=s["i"], lam=s["lam"], dy=dy, h0=s["h0"])
    for bad in (dict(dy=None), dict(dy=dy[:1]), dict(dy=dy.float()), dict(dh_final=torch.zeros(2, 7, device="cuda")),
                dict(kept=torch.zeros(3, 8, device="cuda")), dict(kept=torch.zeros(2, 8, device="cuda").half())):
        with pytest.raises(ValueError):
            layer.lru_backward(**(args | bad))
    with pytest.raises(GdrError) as e:
        layer.lru_backward(**args, workspace=torch.empty(16, device="cuda"))
    assert e.value.status == 5
