"""The gradient of the selective state space scan against the reverse recurrence in 64 bits and against differences.

Tolerances.  Every term is a product of a state, a state's gradient and a few inputs; both chains carry the forward's
error of 2e-5 of their terms (test_gpu_ssm.py), so gradients are held to 5e-5 of the sum of their terms' sizes, and
16-bit ones to half a unit in the last place on top.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, layer
from ssm_reference import scan, scan_backward
from test_gpu_ssm import HALF_ULP, LENGTHS, TYPES, make

pytestmark = pytest.mark.gpu
TOL = 5e-5
TOKENS = ("x", "dt", "z", "B", "C")


def reference(s, rows, dy, dh_final, i, softplus=True):
    p = {k: (None if s[k] is None else s[k][rows]) for k in TOKENS}
    return scan_backward(p["x"], p["dt"], s["A"], p["B"], p["C"], dy[rows], s["D"], p["z"], s["dt_bias"],
                         None if s["h0"] is None else s["h0"][i], None if dh_final is None else dh_final[i], softplus)


def compare(s, rows_of, dy, dh_final, got, io, softplus=True):
    """rows_of: the leading index of each sequence's tokens."""
    sums = {}
    for i, rows in enumerate(rows_of):
        want = reference(s, rows, dy, dh_final, i, softplus)
        for name in ("dx", "ddt", "dB", "dC", "dz", "dh0"):
            have = getattr(got, name)
            if have is None:
                continue
            v, size = want[name]
            have = have[i] if name == "dh0" else have[rows]
            ulp = 0.0 if name == "dh0" else HALF_ULP[io]
            err = (have.double() - v).abs()
            assert bool((err <= TOL * size + ulp * v.abs() + 2.0 ** -24).all()), (name, i, float(err.max()))
        for name in ("dA", "dD", "ddt_bias"):
            if name in want:
                v, size = sums.get(name, (0, 0))
                sums[name] = (v + want[name][0], size + want[name][1])
    for name, (v, size) in sums.items():
        if getattr(got, name) is not None:
            err = (getattr(got, name).double() - v).abs()
            assert bool((err <= TOL * size + 1e-30).all()), (name, float((err / size.clamp_min(1e-30)).max()))


def randn(*shape, io=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(io).cuda()


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("B,T,D,N,G,pad,parts", [
    (1, 1, 1, 1, 1, 0, ("Dk", "z", "bias", "h0")), (2, 3, 5, 3, 1, 1, ("z", "h0")), (1, 17, 64, 8, 2, 0, ("bias",)),
    (2, 64, 130, 12, 2, 2, ("Dk", "bias", "h0")), (1, 65, 256, 16, 1, 8, ("Dk", "z", "bias", "h0")),
    (3, 130, 96, 16, 4, 0, ("Dk", "z", "bias")), (2, 100, 72, 32, 3, 8, ("z", "bias", "h0")),
    (1, 300, 40, 64, 1, 0, ("Dk", "z", "bias", "h0")), (1, 700, 264, 20, 1, 0, ("Dk", "z", "bias", "h0")),
    (2, 1000, 8, 5, 8, 0, ("bias", "h0")), (9, 40, 4104, 4, 1, 0, ("Dk", "z", "bias", "h0"))])
def test_batches(B, T, D, N, G, pad, parts, io):
    s = make((B, T), D, N, G, io, pad=pad, parts=parts)
    dy = randn(B, T, D, io=io, seed=1)
    dh = randn(B, D, N, seed=2) if "h0" in parts else None
    got = layer.ssm_backward(**s, dy=dy, dh_final=dh)
    for name, part in (("dD", "Dk"), ("dz", "z"), ("ddt_bias", "bias"), ("dh0", "h0")):
        assert (getattr(got, name) is not None) == (part in parts)
    compare(s, range(B), dy, dh, got, io)
    again = layer.ssm_backward(**s, dy=dy, dh_final=dh)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,N,G", [(40, 16, 1), (264, 12, 2), (65, 33, 1), (24, 7, 3)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, D, N, G, io):
    s = make((sum(lens),), D, N, G, io, n=len(lens))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    dy, dh = randn(sum(lens), D, io=io, seed=1), randn(len(lens), D, N, seed=2)
    got = layer.ssm_backward(**s, dy=dy, dh_final=dh, cu_seqlens=cu)
    rows, at = [], 0
    for n in lens:
        rows.append(slice(at, at + n))
        at += n
    compare(s, rows, dy, dh, got, io)


def test_a_sequence_does_not_see_its_neighbours():
    lens = [100, 90, 200]
    s = make((390,), 72, 16, 1, torch.float32, n=3)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    dy = randn(390, 72, seed=1)
    got = layer.ssm_backward(**s, dy=dy, cu_seqlens=cu)
    bad = {k: (v.clone() if k in (*TOKENS, "h0") else v) for k, v in s.items()}
    for t in (*(bad[k] for k in TOKENS), dy):
        t[:100], t[190:] = float("nan"), float("inf")
    bad["h0"][0] = float("nan")
    out = layer.ssm_backward(**bad, dy=dy, cu_seqlens=cu)
    for name in ("dx", "ddt", "dB", "dC", "dz"):
        assert torch.equal(getattr(got, name)[100:190], getattr(out, name)[100:190]), name
    assert torch.equal(got.dh0[1], out.dh0[1])


def test_steps_without_softplus():
    s = make((1, 40), 16, 8, 1, torch.float32, parts=("h0", "z"))
    s["dt"] = torch.rand(1, 40, 16, device="cuda")
    dy = randn(1, 40, 16, seed=1)
    compare(s, [0], dy, None, layer.ssm_backward(**s, dy=dy, softplus=False), torch.float32, softplus=False)


def test_a_batch_that_fills_the_gpu_is_walked_whole():
    s = make((8, 100), 4096, 16, 1, torch.bfloat16, n=8)      # 512 blocks of 64 channels
    dy = randn(8, 100, 4096, io=torch.bfloat16, seed=1)
    compare(s, range(8), dy, None, layer.ssm_backward(**s, dy=dy), torch.bfloat16)


def test_against_differences():
    s = make((1, 6), 4, 3, 2, torch.float32)
    dy, dh = randn(1, 6, 4, seed=1), randn(1, 4, 3, seed=2)
    got = layer.ssm_backward(**s, dy=dy, dh_final=dh)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="ddt_bias", h0="dh0")

    def loss(v):
        y, h, *_ = scan(v["x"][0], v["dt"][0], v["A"], v["B"][0], v["C"][0], v["D"], v["z"][0], v["dt_bias"], v["h0"][0])
        return float((y * dy[0].double()).sum() + (h * dh[0].double()).sum())

    base, h = {k: v.double() for k, v in s.items()}, 1e-5
    for key, name in names.items():
        grad = getattr(got, name).reshape(-1)
        for i in range(0, base[key].numel(), 3):
            hi, lo = ({k: v.clone() for k, v in base.items()} for _ in range(2))
            hi[key] = hi[key].contiguous()
            lo[key] = lo[key].contiguous()
            hi[key].view(-1)[i] += h
            lo[key].view(-1)[i] -= h
            assert float(grad[i]) == pytest.approx((loss(hi) - loss(lo)) / (2 * h), rel=1e-4, abs=1e-4), (key, i)


def test_another_stream():
    side = torch.cuda.Stream()
    s = make((1, 3000), 256, 16, 1, torch.bfloat16)
    dy = randn(1, 3000, 256, io=torch.bfloat16, seed=1)
    side.wait_stream(torch.cuda.current_stream())
    got = layer.ssm_backward(**s, dy=dy, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, layer.ssm_backward(**s, dy=dy)))


def test_refusals():
    s = make((2, 5), 8, 4, 2, torch.bfloat16)
    dy = randn(2, 5, 8, io=torch.bfloat16)
    for bad in (dict(dy=dy[:1]), dict(dy=dy.float()), dict(dh_final=torch.zeros(2, 8, 3, device="cuda")),
                dict(B=s["B"].float()), dict(h0=s["h0"][:1])):
        with pytest.raises(ValueError):
            layer.ssm_backward(**({**s, "dy": dy} | bad))
    with pytest.raises(GdrError) as e:
        layer.ssm_backward(**s, dy=dy, workspace=torch.empty(16, device="cuda"))
    assert e.value.status == 5
