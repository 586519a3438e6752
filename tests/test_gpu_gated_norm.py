"""The gated norm of a recurrence's output, and its gradient, against the definition in 64 bits.

Tolerances.  The sum of up to 8192 squares has only positive terms and a tree of depth at most 26: 1.6e-6 of itself, half of
it after the root; the gate is off by 2^-21 of itself (the hardware's 2^x and reciprocal) and a handful of products follow:
under 1e-5 of the sizes of a value's terms.  16-bit outputs have half a unit in the last place on top.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, layer

pytestmark = pytest.mark.gpu
EPS = 1e-6
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SHAPES = [(1, 1, 1), (3, 2, 7), (5, 1, 64), (700, 3, 128), (33, 16, 128), (2, 32, 128), (1300, 5, 100), (40, 7, 33),
          (9, 2, 256), (50, 4, 250), (70, 1, 512), (30, 3, 1000), (20, 2, 1024), (9, 2, 2050), (40, 1, 4096), (7, 1, 8192),
          (3, 300, 64), (2, 20000, 16), (11, 24, 8), (6, 4, 8191), (300, 48, 128)]


def make(tokens, H, V, io, per_head=False, seed=0, pad=None):
    gen = torch.Generator().manual_seed(seed)

    def wide(scale):
        p = 0 if pad is None else pad
        return (scale * torch.randn(tokens, H * V + 2 * p, generator=gen)).to(io).cuda()[:, p:p + H * V].unflatten(1, (H, V))

    w = (1 + 0.1 * torch.randn(*((H, V) if per_head else (V,)), generator=gen)).to(io).cuda()
    return wide(0.3), wide(2.0), w


def gate_of(z, gate):
    """The gate, its slope, and the size of the slope's terms."""
    sig, z = torch.sigmoid(z.double()), z.double()
    if gate == "sigmoid":
        return sig, sig * torch.sigmoid(-z), sig * torch.sigmoid(-z) + 2.0 ** -22 * sig
    return z * sig, sig + z * sig * torch.sigmoid(-z), sig * (1 + z.abs())


def check(y, x, z, w, gate, io):
    f, _, _ = gate_of(z, gate)
    x = x.double()
    want = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double() * f
    err = (y.double() - want).abs()
    assert y.dtype == io
    assert bool((err <= (1e-5 + HALF_ULP[io]) * want.abs() + 2.0 ** -24).all()), float(err.max())


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("tokens,H,V", SHAPES)
def test_forward(tokens, H, V, per_head, gate, io):
    x, z, w = make(tokens, H, V, io, per_head)
    check(layer.gated_norm_forward(x, z, w, gate=gate, eps=EPS), x, z, w, gate, io)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("pad", [1, 2, 8])
@pytest.mark.parametrize("tokens,H,V", [(6, 4, 128), (5, 3, 33), (6, 2, 1000), (4, 1, 2050), (3, 2, 4)])
def test_slices(tokens, H, V, pad, io):
    x, z, w = make(tokens, H, V, io, True, pad=pad)
    check(layer.gated_norm_forward(x, z, w, eps=EPS), x, z, w, "silu", io)
    backward_check(x, z, w, "silu", io)
    lead = layer.gated_norm_forward(x[None], z[None], w, eps=EPS)         # more leading dimensions
    assert lead.shape == (1, tokens, H, V) and torch.equal(lead[0], layer.gated_norm_forward(x, z, w, eps=EPS))
    t = torch.randn(V, H, tokens, device="cuda").to(io).permute(2, 1, 0)   # no one stride: copied
    check(layer.gated_norm_forward(t, z, w, eps=EPS), t, z, w, "silu", io)


def backward_check(x, z, w, gate, io):
    tokens, H, V = x.shape
    gen = torch.Generator().manual_seed(77)
    dy = torch.randn(tokens, H, V, generator=gen).to(io).cuda()
    dx, dz, dw = layer.gated_norm_backward(dy, x, z, w, gate=gate, eps=EPS)
    f, slope, ssize = gate_of(z, gate)
    x64, g, w64 = x.double(), dy.double(), w.double()
    rstd = 1 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + EPS)
    n, dn = x64 * rstd, g * w64 * f
    want = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    size = rstd * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True))
    err = (dx.double() - want).abs()
    assert bool((err <= 1e-5 * size + HALF_ULP[io] * want.abs() + 2.0 ** -24).all()), ("dx", float((err / size).max()))
    want = g * n * w64 * slope
    err = (dz.double() - want).abs()
    assert bool((err <= 1e-5 * (g * n * w64).abs() * ssize + HALF_ULP[io] * want.abs() + 2.0 ** -24).all()), \
        ("dz", float(err.max()))
    terms = g * n * f
    dims = 0 if w.dim() == 2 else (0, 1)
    # a column's sum: at most 80 rows a thread, 320 partial sums in turn and 5 levels, 20 roundings a term: 425 x 2^-24
    err = (dw.double() - terms.sum(dims)).abs()
    assert dw.shape == w.shape and dw.dtype == torch.float32
    assert bool((err <= 2.6e-5 * terms.abs().sum(dims) + 1e-30).all()), ("dw", float(err.max()))
    again = layer.gated_norm_backward(dy, x, z, w, gate=gate, eps=EPS)
    assert torch.equal(dx, again[0]) and torch.equal(dz, again[1]) and torch.equal(dw, again[2])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("tokens,H,V", SHAPES)
def test_backward(tokens, H, V, per_head, gate, io):
    backward_check(*make(tokens, H, V, io, per_head), gate, io)


@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_backward_against_differences(gate):
    x, z, w = (t.double() for t in make(2, 3, 20, torch.float32, True))
    dy = torch.randn(2, 3, 20, generator=torch.Generator().manual_seed(3)).cuda()
    got = layer.gated_norm_backward(dy, x.float(), z.float(), w.float(), gate=gate, eps=EPS)

    def loss(x, z, w):
        return float((dy.double() * x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w * gate_of(z, gate)[0]).sum())

    h, base = 1e-5, [x, z, w]
    for k, grad in enumerate(got):
        for j in range(0, base[k].numel(), 7):
            hi, lo = ([t.clone().contiguous() for t in base] for _ in range(2))
            hi[k].view(-1)[j] += h
            lo[k].view(-1)[j] -= h
            assert float(grad.reshape(-1)[j]) == pytest.approx((loss(*hi) - loss(*lo)) / (2 * h), rel=1e-4, abs=1e-4)


def test_rows_of_zeros_infinities_and_nan():
    x, z, w = make(6, 2, 128, torch.float32)
    clean = layer.gated_norm_forward(x, z, w)
    x[1, 0], x[2, 1, 5], z[3, 0, 7], z[4, 1, 9] = 0, float("nan"), float("inf"), -float("inf")
    x[5, 1, 3] = float("inf")
    y = layer.gated_norm_forward(x, z, w, gate="sigmoid")
    assert not y[1, 0].any() and bool(y[2, 1].isnan().all()) and bool(y[5, 1, 3].isnan())
    assert bool(y[3].isfinite().all()) and float(y[4, 1, 9]) == 0.0
    again = layer.gated_norm_forward(x, z, w)
    for row, head in ((0, 0), (0, 1), (1, 1), (2, 0), (3, 1), (4, 0), (5, 0)):
        assert torch.equal(again[row, head], clean[row, head])
    dy = torch.ones_like(x)
    dx, dz, _ = layer.gated_norm_backward(dy, x, z, w, gate="sigmoid")
    assert bool(dx[1, 0].isfinite().all()) and not dz[1, 0].any() and float(dz[3, 0, 7]) == 0.0 == float(dz[4, 1, 9])


def test_no_tokens():
    x, w = torch.empty(0, 4, 64, device="cuda"), torch.ones(4, 64, device="cuda")
    assert layer.gated_norm_forward(x, x, w).shape == (0, 4, 64)
    dx, dz, dw = layer.gated_norm_backward(x, x, x, w)
    assert dx.shape == dz.shape == (0, 4, 64) and dw.shape == (4, 64) and not dw.any()


def test_another_stream():
    side = torch.cuda.Stream()
    x, z, w = make(3000, 16, 128, torch.bfloat16, pad=8)
    side.wait_stream(torch.cuda.current_stream())
    y = layer.gated_norm_forward(x, z, w, stream=side)
    got = layer.gated_norm_backward(y, x, z, w, stream=side)
    side.synchronize()
    assert torch.equal(y, layer.gated_norm_forward(x, z, w))
    assert all(torch.equal(a, b) for a, b in zip(got, layer.gated_norm_backward(y, x, z, w)))


def test_offsets_beyond_32_bits():
    T, H, V = 530_000, 32, 128                            # 2.17e9 elements
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, H, V, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(V, generator=gen, device="cuda", dtype=torch.bfloat16)
    y = layer.gated_norm_forward(x, x, w)
    last = layer.gated_norm_forward(x[-300:], x[-300:], w)
    assert torch.equal(y[-300:], last)
    dx, dz, _ = layer.gated_norm_backward(y, x, x, w)
    dx2, dz2, _ = layer.gated_norm_backward(last, x[-300:], x[-300:], w)
    assert torch.equal(dx[-300:], dx2) and torch.equal(dz[-300:], dz2)


def test_refusals():
    x, z, w = make(4, 2, 64, torch.bfloat16)
    for bad in (dict(z=None), dict(z=z[:3]), dict(z=z.float()), dict(weight=w[:32]), dict(weight=w.float()),
                dict(weight=torch.ones(3, 64, device="cuda", dtype=torch.bfloat16)), dict(weight=None), dict(gate="relu"),
                dict(gate=None), dict(x=x.cpu()), dict(x=x[0, 0], z=z[0, 0])):
        args = dict(x=x, z=z, weight=w) | bad
        with pytest.raises(ValueError):
            layer.gated_norm_forward(**args)
        with pytest.raises(ValueError):
            layer.gated_norm_backward(x, **args)
    for eps in (float("nan"), -1.0, float("inf")):
        with pytest.raises(GdrError) as e:
            layer.gated_norm_forward(x, z, w, eps=eps)
        assert e.value.status == 9
    big = torch.zeros(1, 1, 8193, device="cuda")
    with pytest.raises(GdrError) as e:
        layer.gated_norm_forward(big, big, big[0, 0])
    assert e.value.status == 2
    for bad in (None, x.float(), x[:2]):
        with pytest.raises(ValueError):
            layer.gated_norm_backward(bad, x, z, w)
    with pytest.raises(GdrError) as e:
        layer.gated_norm_backward(x, x, z, w, workspace=torch.empty(1, device="cuda", dtype=torch.uint8))
    assert e.value.status == 5


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("tokens,H,V", [(2600, 3, 33), (1, 1, 9), (9000, 1, 100), (701, 7, 251), (400, 5, 1001), (50, 1, 8180)])
def test_rows_between_boundaries(tokens, H, V, per_head, io):
    """All tensors' rows lie alike between 16-byte boundaries, the gate's in a wider row; what lies beside it is not seen."""
    x, _, w = make(tokens, H, V, io, per_head, seed=5)
    gen = torch.Generator().manual_seed(6)
    z = torch.full((tokens, H * V + 24), float("nan")).to(io)
    z[:, :H * V] = 2 * torch.randn(tokens, H * V, generator=gen)
    z = z.cuda()[:, :H * V].unflatten(1, (H, V))
    check(layer.gated_norm_forward(x, z, w), x, z, w, "silu", io)
    backward_check(x, z, w, "silu", io)
