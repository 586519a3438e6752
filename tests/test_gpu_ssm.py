"""The selective state space scan (prompts, packed prompts, single tokens) against the recurrence in 64 bits.

Tolerances.  Every term of a state carries a product of decays exp(Delta A).  Each decay is off by at most 2^-22 of
itself (the hardware's 2^x) beside the rounding of its exponent, and the decays of t tokens multiply; with steps of
0.001 and more and rates of 1 and more a term has lost 1/e after 1000 tokens, so errors reach 1000 * 2^-22 = 2.4e-4 of a
term at the very worst, if all were the same way; their mean is below 1e-8 near 1 (measured), which leaves 1e-5.  States
and fp32 outputs are held to 2e-5 of the sum of their terms' sizes, 16-bit outputs to half a unit on top.
"""
import math

import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, gdr, layer
from ssm_reference import scan

pytestmark = pytest.mark.gpu
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
TOL = 2e-5


def make(lead, D, N, G, io, seed=0, n=None, pad=0, parts=("Dk", "z", "bias", "h0")):
    """Inputs of tokens `lead`; pad: x, z and B, C as slices of wider rows, `pad` elements apart."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen) * scale

    def wide(*cols):
        row = randn(*lead, sum(cols) + pad * len(cols)).to(io).cuda()
        at, out = pad, []
        for c in cols:
            out.append(row[..., at:at + c])
            at += c + pad
        return out

    (x, z), (b, c) = wide(D, D), wide(G * N, G * N)
    step = torch.exp(torch.rand(D, generator=gen) * math.log(100) + math.log(1e-3))
    s = dict(x=x, dt=randn(*lead, D, scale=0.5).to(io).cuda(),
             A=(-torch.arange(1, N + 1) * (0.9 + 0.2 * torch.rand(D, 1, generator=gen))).cuda(),
             B=b.unflatten(-1, (G, N)), C=c.unflatten(-1, (G, N)), D=(1 + 0.1 * randn(D)).cuda(), z=z,
             dt_bias=(step + torch.log(-torch.expm1(-step))).cuda(),
             h0=randn(n or lead[0], D, N).cuda())
    for part, key in (("Dk", "D"), ("z", "z"), ("bias", "dt_bias"), ("h0", "h0")):
        if part not in parts:
            s[key] = None
    return s


def check(s, i, rows, y, h, io, softplus=True):
    """Sequence i, its tokens given by `rows` (an index of the leading dimensions)."""
    pick = lambda t: None if t is None else t[rows]  # noqa: E731
    want, last, _, ysize, sizes = scan(pick(s["x"]), pick(s["dt"]), s["A"], pick(s["B"]), pick(s["C"]), s["D"],
                                       pick(s["z"]), s["dt_bias"], None if s["h0"] is None else s["h0"][i], softplus)
    assert bool(((y[rows].double() - want).abs() <= TOL * ysize + HALF_ULP[io] * want.abs() + 2.0 ** -24).all()), i
    if h is not None:
        assert bool(((h[i].double() - last).abs() <= TOL * sizes[-1] + 1e-30).all()), i


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("B,T,D,N,G,pad,parts", [
    (1, 1, 1, 1, 1, 0, ("Dk", "z", "bias", "h0")), (2, 3, 5, 3, 1, 1, ("z", "h0")), (1, 17, 64, 8, 2, 0, ("bias",)),
    (2, 64, 130, 12, 2, 2, ("Dk", "bias", "h0")), (1, 65, 256, 16, 1, 8, ("Dk", "z", "bias", "h0")),
    (3, 130, 96, 16, 4, 0, ("Dk", "z", "bias")), (2, 100, 72, 32, 3, 8, ("z", "bias", "h0")),
    (1, 300, 40, 64, 1, 0, ("Dk", "z", "bias", "h0")), (1, 700, 264, 20, 1, 0, ("Dk", "z", "bias", "h0")),
    (2, 1000, 8, 5, 8, 0, ("bias", "h0")), (9, 40, 4104, 4, 1, 0, ("Dk", "z", "bias", "h0"))])
def test_batches(B, T, D, N, G, pad, parts, io):
    s = make((B, T), D, N, G, io, pad=pad, parts=parts)
    y, h = layer.ssm_forward(**s)
    for i in range(B):
        check(s, i, i, y, h, io)
    y2, none = layer.ssm_forward(**s, want_h_final=False)
    assert none is None and torch.equal(y, y2)


def test_whole_and_in_segments():
    # a batch that fills the GPU is scanned whole, one sequence of it in segments: two paths, one result within rounding
    s = make((20, 500), 4096, 16, 1, torch.bfloat16, n=20)
    y, h = layer.ssm_forward(**s)
    assert gdr.gdr_last_variant() == "ssm"
    first = {k: (v[:1] if k in ("x", "dt", "z", "B", "C", "h0") else v) for k, v in s.items()}
    y1, h1 = layer.ssm_forward(**first)
    assert gdr.gdr_last_variant() == "ssm_segments"
    assert float((h1 - h[:1]).abs().max()) <= TOL * float(h.abs().max())
    check(s, 0, 0, y, h, torch.bfloat16)
    check(first, 0, 0, y1, h1, torch.bfloat16)


LENGTHS = [[5], [0], [1, 0, 2, 3], [64, 64], [700, 0, 1, 33, 0], [0, 0, 127, 128, 129], [3] * 70]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("D,N,G", [(40, 16, 1), (264, 12, 2), (65, 33, 1), (24, 7, 3)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, D, N, G, io):
    s = make((sum(lens),), D, N, G, io, n=len(lens))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    y, h = layer.ssm_forward(**s, cu_seqlens=cu)
    at = 0
    for i, n in enumerate(lens):
        check(s, i, slice(at, at + n), y, h, io)
        at += n
    s["h0"] = None
    y, h = layer.ssm_forward(**s, cu_seqlens=cu)
    at = 0
    for i, n in enumerate(lens):
        check(s, i, slice(at, at + n), y, h, io)
        at += n


def test_a_sequence_does_not_see_its_neighbours():
    lens = [100, 90, 200]
    s = make((390,), 72, 16, 1, torch.float32, n=3)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    y, h = layer.ssm_forward(**s, cu_seqlens=cu)
    bad = {k: (v.clone() if k in ("x", "dt", "z", "B", "C", "h0") else v) for k, v in s.items()}
    for k in ("x", "dt", "z", "B", "C"):
        bad[k][:100], bad[k][190:] = float("nan"), float("inf")
    bad["h0"][0] = float("nan")
    y2, h2 = layer.ssm_forward(**bad, cu_seqlens=cu)
    assert torch.equal(y[100:190], y2[100:190]) and torch.equal(h[1], h2[1])


@pytest.mark.parametrize("softplus", [True, False])
def test_steps_of_every_size(softplus):
    # raw steps from far below softplus's resolution to far above its threshold; without softplus they are taken as given
    s = make((1, 64), 16, 8, 1, torch.float32, parts=("h0",))
    s["dt"] = torch.linspace(-30, 40, 64 * 16).view(1, 64, 16).cuda() if softplus else torch.rand(1, 64, 16).cuda()
    y, h = layer.ssm_forward(**s, softplus=softplus)
    check(s, 0, 0, y, h, torch.float32, softplus)


def test_long_slow_decay():
    s = make((1, 20000), 8, 16, 1, torch.float32, parts=("h0", "z"))
    s["dt"] = torch.full((1, 20000, 8), -6.9, device="cuda")        # Delta = 0.001
    y, h = layer.ssm_forward(**s)
    check(s, 0, 0, y, h, torch.float32)


def test_the_same_bits_again():
    s = make((1, 5000), 512, 16, 1, torch.bfloat16)
    y, h = layer.ssm_forward(**s)
    for _ in range(3):
        y2, h2 = layer.ssm_forward(**s)
        assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("n,D,N,G,pad,parts", [
    (1, 1, 1, 1, 0, ("Dk", "z", "bias")), (3, 5, 3, 1, 1, ("z",)), (2, 64, 8, 2, 0, ("bias",)),
    (70, 130, 12, 2, 2, ("Dk", "bias")), (5, 257, 16, 1, 8, ("Dk", "z", "bias")), (4, 72, 33, 3, 0, ()),
    (3, 40, 64, 1, 0, ("Dk", "z", "bias"))])
def test_step(n, D, N, G, pad, parts, io):
    pool = n + 5
    s = make((n,), D, N, G, io, n=pool, pad=pad, parts=(*parts, "h0"))
    h = s.pop("h0")
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32).cuda()
    padding = []
    if n > 2:
        padding = [0, n - 1]
        slots[0], slots[n - 1] = -1, pool
        s["x"][0], s["dt"][n - 1] = float("nan"), float("inf")
    before = h.clone()
    y = layer.ssm_step(h=h, slots=slots, **s)
    for i in range(n):
        if i in padding:
            assert not y[i].any()
            continue
        at = int(slots[i])
        one = {k: (v[i:i + 1] if k in ("x", "dt", "z", "B", "C") and v is not None else v) for k, v in s.items()}
        one["h0"] = before[at:at + 1].clone()
        check(one, 0, slice(0, 1), y[i:i + 1], h[at:at + 1], io)
        before[at] = h[at]
    assert torch.equal(before, h)


def test_steps_go_on_from_a_prompt():
    s = make((2, 30), 96, 16, 1, torch.float32)
    whole, last = layer.ssm_forward(**s)
    tokens = ("x", "dt", "z", "B", "C")
    _, h = layer.ssm_forward(**{k: (v[:, :20] if k in tokens else v) for k, v in s.items()})
    rest = {k: v for k, v in s.items() if k != "h0"}
    for t in range(20, 30):
        y = layer.ssm_step(h=h, **{k: (v[:, t] if k in tokens else v) for k, v in rest.items()})
        assert torch.allclose(y, whole[:, t], rtol=1e-4, atol=1e-5)
    assert torch.allclose(h, last, rtol=1e-4, atol=1e-5)


def test_another_stream():
    side = torch.cuda.Stream()
    s = make((1, 4000), 512, 16, 1, torch.bfloat16)
    side.wait_stream(torch.cuda.current_stream())
    y, h = layer.ssm_forward(**s, stream=side)
    side.synchronize()
    assert torch.equal(y, layer.ssm_forward(**s)[0])


def test_refusals():
    s = make((2, 5), 8, 4, 2, torch.bfloat16)
    tok = make((3,), 8, 4, 2, torch.bfloat16, n=3)
    h = tok.pop("h0")
    cu = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    for bad in (dict(x=s["x"][0]), dict(cu_seqlens=cu), dict(dt=s["dt"].float()), dict(A=s["A"].double()),
                dict(A=s["A"][:, :3].contiguous()), dict(B=s["B"][..., :1, :]), dict(C=s["C"].float()),
                dict(D=s["D"][:4]), dict(z=s["z"][:1]), dict(dt_bias=s["dt_bias"].bfloat16()),
                dict(h0=s["h0"].transpose(1, 2)), dict(x=s["x"].cpu())):
        with pytest.raises(ValueError):
            layer.ssm_forward(**(s | bad))
    for bad in (dict(h=h[:, :4]), dict(h=h.double()), dict(slots=torch.zeros(3, device="cuda")), dict(x=s["x"])):
        with pytest.raises(ValueError):
            layer.ssm_step(**({**tok, "h": h} | bad))
    with pytest.raises(GdrError) as e:
        layer.ssm_step(h=h[:2].contiguous(), **tok)               # three rows, two states
    assert e.value.status == 2
    with pytest.raises(GdrError) as e:
        layer.ssm_forward(**make((1, 2), 4, 65, 1, torch.float32))
    assert e.value.status == 2
    with pytest.raises(GdrError) as e:                             # 8 channels in 3 groups
        layer.ssm_forward(**make((1, 2), 8, 4, 3, torch.float32))
    assert e.value.status == 2
    long = make((1, 4000), 64, 16, 1, torch.float32)
    with pytest.raises(GdrError) as e:
        layer.ssm_forward(**long, workspace=torch.empty(16, device="cuda"))
    assert e.value.status == 5
