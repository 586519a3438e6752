"""The layer norm (residual, gradient) against its definition in 64 bits.

Tolerances, with R = rstd mean|s| of a row: the mean is a sum in a tree of depth at most 42 (32 values a thread, 10 levels),
so it is off by at most 42 x 2^-24 = 2.5e-6 of mean|s|, which moves xh by 2.5e-6 R; the squares' sum, the root and a
handful of operations after them stay under 1e-5 of the value.  16-bit outputs have half a unit in the last place on top.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, layer

pytestmark = pytest.mark.gpu
EPS = 1e-5
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SHAPES = [(1, 1), (3, 7), (5, 64), (700, 250), (1, 256), (2, 264), (700, 512), (701, 1000), (33, 1024), (400, 2048),
          (20, 2050), (500, 4096), (16, 4096), (1, 8192), (400, 8200), (2, 16384), (310, 16000), (3, 32768),
          (305, 32768), (400, 2553), (1300, 887), (305, 32761), (4451, 2278)]


def make(rows, D, io, seed=0, ld=None, mean=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, ld or D, generator=gen).to(io).cuda()[:, :D]
    res = (2 * torch.randn(rows, D, generator=gen) + mean * torch.randn(rows, 1, generator=gen)).to(io).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=gen)).to(io).cuda()
    b = (0.1 * torch.randn(D, generator=gen)).to(io).cuda()
    return x, res, w, b


def parts(s):
    """xh, rstd and R of rows in 64 bits."""
    m = s.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((s - m) ** 2).mean(-1, keepdim=True) + EPS)
    return (s - m) * rstd, rstd, rstd * s.abs().mean(-1, keepdim=True)


def check(y, s, w, b, io):
    xh, rstd, R = parts(s)
    w = w.double()
    want = xh * w + (b.double() if b is not None else 0)
    # the sum s itself is rounded to 2^-24 of its size; a bias adds one rounding
    tol = 1e-5 * (xh * w).abs().amax(-1, keepdim=True) + (3e-6 * R + 2.0 ** -23 * rstd * s.abs()) * w.abs()
    err = (y.double() - want).abs()
    assert bool((err <= tol + (HALF_ULP[io] + 2.0 ** -24) * want.abs() + 2.0 ** -24).all()), float(err.max())


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("rows,D", SHAPES)
def test_forward(rows, D, io):
    x, res, w, b = make(rows, D, io)
    y, r = layer.layernorm_forward(x, w, b, res, eps=EPS)
    check(y, x.double() + res.double(), w, b, io)
    assert torch.equal(r, (x.float() + res.float()).to(io))
    y, r = layer.layernorm_forward(x, w, eps=EPS)
    check(y, x.double(), w, None, io)
    assert r is x
    none, r = layer.layernorm_forward(x, w, b, res, want_y=False)
    assert none is None and torch.equal(r, (x.float() + res.float()).to(io))


def test_a_mean_far_from_zero():
    """fp32 rows whose mean is 1000 times their spread: one pass over squares would leave nothing of it."""
    x, res, w, b = make(40, 4096, torch.float32, mean=0.0)
    x += 2000
    y, _ = layer.layernorm_forward(x, w, b, res, eps=EPS)
    check(y, x.double() + res.double(), w, b, torch.float32)
    xh, _, _ = parts(x.double() + res.double())
    assert float((y.double() - xh * w.double() - b.double()).abs().max()) < 6e-3      # 2.5e-6 R with R = 890, and 5 widths


def test_rows_of_one_value_infinities_and_nan():
    x, _, w, b = make(5, 512, torch.float32, seed=2)
    clean, _ = layer.layernorm_forward(x, w, b)
    x[1] = 7.0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    y, _ = layer.layernorm_forward(x, w, b)
    assert torch.equal(y[[0, 2]], clean[[0, 2]])
    assert torch.equal(y[1], b)                              # nothing varies
    assert bool(y[3].isnan().all()) and bool(y[4].isnan().all())


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,ld", [(64, 192), (250, 251), (8, 24), (4096, 8200), (2048, 2049)])
def test_slices_and_leading_dimensions(D, ld, io):
    x, res, w, b = make(6, D, io, seed=4, ld=ld)
    wide = torch.empty(6, ld + 3, device="cuda", dtype=io)
    wide[:, 3:3 + D] = res
    y, r = layer.layernorm_forward(x.unflatten(0, (2, 3)), w, b, wide[:, 3:3 + D].unflatten(0, (2, 3)), eps=EPS)
    assert y.shape == (2, 3, D)
    check(y.flatten(0, 1), x.double() + res.double(), w, b, io)
    assert torch.equal(r.flatten(0, 1), (x.float() + res.float()).to(io))
    t = torch.randn(D, 6, device="cuda").to(io).t()           # no one stride: copied
    check(layer.layernorm_forward(t, w, b, eps=EPS)[0], t.double(), w, b, io)


def backward_check(rows, D, io, with_dr):
    r, dy, w, _ = make(rows, D, io, seed=5)
    dr = make(rows, D, io, seed=6)[0].contiguous() if with_dr else None
    dx, dw, db = layer.layernorm_backward(dy, r, w, dr, eps=EPS)
    xh, rstd, R = parts(r.double())
    g = dy.double()
    t = g * w.double()
    dot, flat = (t * xh).mean(-1, keepdim=True), t.mean(-1, keepdim=True)
    want = rstd * (t - flat - xh * dot) + (dr.double() if with_dr else 0)
    # dx's terms; xh, off by 2.5e-6 R, multiplies mean|t xh| and, within that mean, |xh| multiplies mean|t|
    size = rstd * (t.abs() + (1 + xh.abs()) * (t.abs().mean(-1, keepdim=True) + (t * xh).abs().mean(-1, keepdim=True)))
    size = size * (1 + R) + (dr.double().abs() if with_dr else 0)
    err = (dx.double() - want).abs()
    assert bool((err <= 1e-5 * size + HALF_ULP[io] * want.abs() + 2.0 ** -24).all()), float((err / size).max())
    # a column's sums: at most 6 rows a thread, 160 partial sums in turn and 5 levels, 40 roundings a term: 211 x 2^-24
    err = (dw.double() - (g * xh).sum(0)).abs()
    assert bool((err <= 1.3e-5 * (g * xh).abs().sum(0) + 3e-6 * (g.abs() * R).sum(0) + 1e-30).all()), float(err.max())
    assert bool(((db.double() - g.sum(0)).abs() <= 1.1e-5 * g.abs().sum(0) + 1e-30).all())
    again = layer.layernorm_backward(dy, r, w, dr, eps=EPS)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and torch.equal(db, again[2])


@pytest.mark.parametrize("with_dr", [False, True])
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("rows,D", SHAPES)
def test_backward(rows, D, io, with_dr):
    backward_check(rows, D, io, with_dr)


# many rows, which come through shared memory: each number of threads a row, whole and odd rows, more rows than places
MANY = [(12000, 256), (11001, 128), (12345, 131), (8000, 512), (6000, 1000), (5001, 1027), (2800, 2048), (3001, 2050),
        (2500, 4096), (2600, 4089), (1000, 8192), (1001, 8191), (700, 16384), (701, 16379), (4000, 2044)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("rows,D", MANY)
def test_many_rows(rows, D, io):
    test_forward(rows, D, io)
    backward_check(rows, D, io, True)
    backward_check(rows, D, io, False)


@pytest.mark.parametrize("io", TYPES)
def test_many_rows_of_a_slice(io):
    x, res, w, b = make(3000, 2048, io, ld=2048 + 64)
    y, r = layer.layernorm_forward(x, w, b, res, eps=EPS)
    whole = layer.layernorm_forward(x.contiguous(), w, b, res, eps=EPS)
    assert torch.equal(y, whole[0]) and torch.equal(r, whole[1])
    check(y, x.double() + res.double(), w, b, io)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("D", range(1, 20))
def test_narrow_rows(D, io):
    """Rows of 1 to 19 columns: the tensors' last vectors hold the ends of several rows."""
    for rows in (1, 2, 5, 13, 600, 2433, 5000):
        test_forward(rows, D, io)
        backward_check(rows, D, io, rows % 2 == 1)


def test_backward_against_differences():
    r, dy, w, _ = make(3, 40, torch.float32, seed=7)
    dx, dw, db = layer.layernorm_backward(dy, r, w, eps=EPS)
    r64, w64, h = r.double(), w.double(), 1e-4

    def loss(r_, w_, b_):
        return float((dy.double() * (parts(r_)[0] * w_ + b_)).sum())

    zero = torch.zeros_like(w64)
    for i, j in ((0, 0), (1, 17), (2, 39)):
        e, f = torch.zeros_like(r64), torch.zeros_like(w64)
        e[i, j] = f[j] = h
        for got, hi, lo in ((dx[i, j], (r64 + e, w64, zero), (r64 - e, w64, zero)),
                            (dw[j], (r64, w64 + f, zero), (r64, w64 - f, zero)), (db[j], (r64, w64, f), (r64, w64, -f))):
            assert float(got) == pytest.approx((loss(*hi) - loss(*lo)) / (2 * h), rel=1e-4, abs=1e-5)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("rows,D", [(7, 33), (700, 250), (1300, 887), (1300, 2133), (700, 4089), (700, 4096), (6000, 1027),
                                    (3001, 4089), (12000, 264)])
def test_a_row_does_not_see_its_neighbours(rows, D, io):
    """Rows that share an aligned vector with their neighbours' ends, which hold NaN and infinity."""
    gen = torch.Generator().manual_seed(rows)
    x, res, dy = (torch.randn(rows, D, generator=gen).to(io).cuda() for _ in range(3))
    w = torch.randn(D, generator=gen).to(io).cuda()
    y, r = layer.layernorm_forward(x, w, w, res)
    dx = layer.layernorm_backward(dy, r, w)[0]
    bad = torch.arange(rows, device="cuda") % 3 == 1
    x[bad], dy[bad] = float("nan"), float("inf")
    y2, r2 = layer.layernorm_forward(x, w, w, res)
    assert torch.equal(y[~bad], y2[~bad]) and torch.equal(r[~bad], r2[~bad]) and bool(y2[bad].isnan().all())
    assert torch.equal(dx[~bad], layer.layernorm_backward(dy, r2, w)[0][~bad])


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, r = layer.layernorm_forward(x, w, w, x)
    assert y.shape == r.shape == (0, 64)
    dx, dw, db = layer.layernorm_backward(x, x, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_another_stream():
    side = torch.cuda.Stream()
    x, res, w, b = make(4000, 2048, torch.bfloat16, seed=8)
    side.wait_stream(torch.cuda.current_stream())
    y, r = layer.layernorm_forward(x, w, b, res, stream=side)
    got = layer.layernorm_backward(y, r, w, stream=side)
    side.synchronize()
    assert torch.equal(y, layer.layernorm_forward(x, w, b, res)[0])
    assert all(torch.equal(a, c) for a, c in zip(got, layer.layernorm_backward(y, r, w)))


def test_offsets_beyond_32_bits():
    rows, D = 66_000, 32768                               # 2.16e9 elements
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(rows, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(D, generator=gen, device="cuda", dtype=torch.bfloat16)
    y, r = layer.layernorm_forward(x, w, w, x)
    y2, r2 = layer.layernorm_forward(x[-400:], w, w, x[-400:])
    assert torch.equal(y[-400:], y2) and torch.equal(r[-400:], r2)
    del r, r2
    dx = layer.layernorm_backward(y, x, w)[0]
    assert torch.equal(dx[-400:], layer.layernorm_backward(y2, x[-400:], w)[0])


def test_refusals():
    x, res, w, b = make(4, 64, torch.bfloat16)
    for bad in (dict(residual=res.float()), dict(residual=res[:3]), dict(weight=w[:32]), dict(weight=w.float()),
                dict(weight=None), dict(bias=b[:32]), dict(bias=b.float()), dict(x=x.cpu()), dict(x=x.double())):
        with pytest.raises(ValueError):
            layer.layernorm_forward(**(dict(x=x, weight=w, bias=b, residual=res) | bad))
    for kw, status in ((dict(eps=float("nan")), 9), (dict(eps=-1.0), 9), (dict(want_y=False), 1)):
        with pytest.raises(GdrError) as e:
            layer.layernorm_forward(x, w, **kw)
        assert e.value.status == status
    big = torch.zeros(1, 32769, device="cuda")
    with pytest.raises(GdrError) as e:
        layer.layernorm_forward(big, big[0])
    assert e.value.status == 2
    for bad in (dict(dy=None), dict(dy=x.float()), dict(d_r=x[:2]), dict(weight=None)):
        with pytest.raises(ValueError):
            layer.layernorm_backward(**(dict(dy=x, r=x, weight=w) | bad))
    with pytest.raises(GdrError) as e:
        layer.layernorm_backward(x, x, w, workspace=torch.empty(1, device="cuda", dtype=torch.uint8))
    assert e.value.status == 5
