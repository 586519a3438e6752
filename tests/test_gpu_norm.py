"""The root-mean-square norm (residual, 8-bit output, gradient) against its definition in 64 bits.

Tolerances.  Sums of up to 32768 fp32 squares in a tree of depth <= 20 and a handful of fp32 operations after them:
relative error well under 1e-5 before the last rounding, so fp32 outputs are held to 1e-5 of the largest value of
their row, 16-bit outputs to half a unit in their last place on top (2^-8 bf16, 2^-11 fp16).  An e4m3 value is within
1/16 of a real one above its smallest normal (2^-6) and within 2^-10 below it.
"""
import numpy as np
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, layer

pytestmark = pytest.mark.gpu
EPS = 1e-6
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(rows, D, io, seed=0, ld=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, ld or D, generator=gen).to(io).cuda()[:, :D]
    res = (2 * torch.randn(rows, D, generator=gen)).to(io).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=gen)).to(io).cuda()
    return x, res, w


def reference(x, res, w):
    s = x.double() + (res.double() if res is not None else 0)
    return s, s / torch.sqrt((s * s).mean(-1, keepdim=True) + EPS) * w.double()


def close(got, want, io):
    err = (got.double() - want).abs()
    top = want.abs().amax(-1, keepdim=True)
    tiny = 2.0 ** -24 if io == torch.float16 else 0.0      # fp16's subnormals
    assert bool((err <= 1e-5 * top + HALF_ULP[io] * want.abs() + tiny).all()), float((err / top.clamp_min(1e-30)).max())


SHAPES = [(1, 1), (3, 7), (5, 64), (700, 250), (1, 256), (2, 264), (700, 512), (701, 1000), (33, 1024), (400, 2048),
          (20, 2050), (500, 4096), (16, 4096), (1, 8192), (400, 8200), (2, 16384), (310, 16000), (3, 32768),
          (305, 32768)]


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_forward(rows, D, io):
    x, res, w = make(rows, D, io)
    y, r, y8, scales = layer.norm_forward(x, w, res, eps=EPS)
    s, want = reference(x, res, w)
    assert y8 is None and scales is None
    close(y, want, io)
    assert torch.equal(r, (x.float() + res.float()).to(io))
    y, r, _, _ = layer.norm_forward(x, w, eps=EPS)
    close(y, reference(x, None, w)[1], io)
    assert r is x


@pytest.mark.parametrize("quant", ["row", 32, 64, 128])
@pytest.mark.parametrize("rows,D,io", [(3, 7, torch.float32), (2, 40, torch.bfloat16), (9, 250, torch.bfloat16),
                                       (700, 512, torch.float16), (400, 1000, torch.float32), (16, 4096, torch.bfloat16),
                                       (400, 4096, torch.bfloat16), (2, 8200, torch.float16), (2, 32768, torch.float32)])
def test_eight_bits(rows, D, io, quant):
    x, res, w = make(rows, D, io, seed=1)
    y, r, y8, scales = layer.norm_forward(x, w, res, eps=EPS, quant=quant)
    _, want = reference(x, res, w)
    close(y, want, io)
    group = D if quant == "row" else quant
    assert scales.shape == (rows, -(-D // group)) and y8.shape == (rows, D)
    pad = torch.nn.functional.pad(want, (0, -D % group)).unflatten(-1, (-1, group))
    amax = pad.abs().amax(-1)
    assert torch.allclose(scales.double(), (amax / 448).clamp_min(2.0 ** -126), rtol=1e-5, atol=0)
    per = scales.double().repeat_interleave(group, 1)[:, :D]
    unit = want / per                                        # what y8 stands for
    assert bool(((y8.double() - unit).abs() <= unit.abs() * (2.0 ** -4 + 1e-4) + 2.0 ** -10).all())


def test_rows_of_zeros_infinities_and_nan():
    x, _, w = make(6, 512, torch.float32, seed=2)
    x[1] = 0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5] = 1e-30
    y, _, y8, scales = layer.norm_forward(x, w, eps=EPS, quant="row")
    keep = [0, 2]
    close(y[keep], reference(x, None, w)[1][keep], torch.float32)
    assert not y[1].any() and not y8[1].float().any() and float(scales[1]) == pytest.approx(2.0 ** -126)
    assert bool(y[3, 5].isnan()) and not y[3, :5].any() and bool(scales[3].isnan())
    assert bool(y[4].isnan().all()) and bool(scales[4].isnan()) and bool(y8[4].float().isnan().all())
    assert bool(y[5].isfinite().all()) and float(y[5].abs().max()) < 1e-24


def test_no_eps_scales_out():
    # with eps = 0 the norm does not depend on the size of the row
    x, _, w = make(4, 300, torch.float32, seed=3)
    y, _, _, _ = layer.norm_forward(x, w, eps=0.0)
    z, _, _, _ = layer.norm_forward(x * 1024, w, eps=0.0)
    assert torch.allclose(y, z, rtol=1e-6, atol=0)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,ld", [(64, 192), (250, 251), (8, 24), (4096, 8200)])
def test_slices_and_leading_dimensions(D, ld, io):
    x, res, w = make(6, D, io, seed=4, ld=ld)
    wide = torch.empty(6, ld + 3, device="cuda", dtype=io)
    wide[:, 3:3 + D] = res
    y, r, _, _ = layer.norm_forward(x.unflatten(0, (2, 3)), w, wide[:, 3:3 + D].unflatten(0, (2, 3)), eps=EPS)
    assert y.shape == (2, 3, D)
    close(y.flatten(0, 1), reference(x, res, w)[1], io)
    assert torch.equal(r.flatten(0, 1), (x.float() + res.float()).to(io))
    # no one stride: copied
    t = torch.randn(D, 6, device="cuda").to(io).t()
    close(layer.norm_forward(t, w, eps=EPS)[0], reference(t, None, w)[1], io)


def backward_reference(dy, r, w, dr):
    r, dy, w = r.double(), dy.double(), w.double()
    rstd = 1 / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS)
    xh = r * rstd
    dx = rstd * (dy * w - xh * (dy * w * xh).mean(-1, keepdim=True)) + (dr.double() if dr is not None else 0)
    return dx, (dy * xh).sum(0)


@pytest.mark.parametrize("with_dr", [False, True])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_backward(rows, D, io, with_dr):
    r, dy, w = make(rows, D, io, seed=5)
    dr = make(rows, D, io, seed=6)[0] if with_dr else None
    dx, dw = layer.norm_backward(dy, r, w, dr, eps=EPS)
    want, want_dw = backward_reference(dy, r, w, dr)
    # dx cancels (D = 1: to nothing); its terms set the scale
    rstd = 1 / torch.sqrt((r.double() ** 2).mean(-1, keepdim=True) + EPS)
    top = (rstd * (dy.double() * w.double()).abs()).amax(-1, keepdim=True) + (dr.double().abs() if with_dr else 0)
    assert bool(((dx.double() - want).abs() <= 1e-5 * top + HALF_ULP[io] * want.abs() + 2.0 ** -24).all())
    # a column's sum of `rows` fp32 products: 1e-6 of the sum of their sizes
    size = (dy.double() * r.double() * rstd).abs().sum(0)
    assert bool(((dw.double() - want_dw).abs() <= 2e-6 * size + 1e-30).all())
    again = layer.norm_backward(dy, r, w, dr, eps=EPS)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_backward_against_differences():
    r, dy, w = make(3, 40, torch.float32, seed=7)
    dx, dw = layer.norm_backward(dy, r, w, eps=EPS)
    r64, w64, h = r.double(), w.double(), 1e-4

    def loss(r_, w_):
        return float((dy.double() * (r_ / torch.sqrt((r_ * r_).mean(-1, keepdim=True) + EPS) * w_)).sum())

    for i, j in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros_like(r64)
        e[i, j] = h
        assert float(dx[i, j]) == pytest.approx((loss(r64 + e, w64) - loss(r64 - e, w64)) / (2 * h), rel=1e-4, abs=1e-5)
        f = torch.zeros_like(w64)
        f[j] = h
        assert float(dw[j]) == pytest.approx((loss(r64, w64 + f) - loss(r64, w64 - f)) / (2 * h), rel=1e-4, abs=1e-5)


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    y, r, y8, scales = layer.norm_forward(x, w, x, quant="row")
    assert y.shape == (0, 64) and scales.shape == (0, 1)
    dx, dw = layer.norm_backward(x, x, w)
    assert dx.shape == (0, 64) and not dw.any()


def test_another_stream():
    side = torch.cuda.Stream()
    x, res, w = make(4000, 2048, torch.bfloat16, seed=8)
    side.wait_stream(torch.cuda.current_stream())
    y, r, _, _ = layer.norm_forward(x, w, res, eps=EPS, stream=side)
    dx, dw = layer.norm_backward(y, r, w, eps=EPS, stream=side)
    side.synchronize()
    assert torch.equal(y, layer.norm_forward(x, w, res, eps=EPS)[0])
    assert torch.equal(dw, layer.norm_backward(y, r, w, eps=EPS)[1])


def test_refusals():
    x, res, w = make(4, 64, torch.bfloat16)
    for bad in (dict(residual=res.float()), dict(residual=res[:3]), dict(weight=w[:32]), dict(weight=w.float()),
                dict(quant="column"), dict(x=x.cpu()), dict(x=x.double())):
        args = dict(x=x, weight=w, residual=res, quant=None) | bad
        with pytest.raises(ValueError):
            layer.norm_forward(args["x"], args["weight"], args["residual"], quant=args["quant"])
    for kw, status in ((dict(quant=48), 9), (dict(eps=float("nan")), 9), (dict(eps=-1.0), 9)):
        with pytest.raises(GdrError) as e:
            layer.norm_forward(x, w, res, **kw)
        assert e.value.status == status
    with pytest.raises(GdrError) as e:      # nothing to write
        layer.norm_forward(x, w, want_y=False)
    assert e.value.status == 1
    big = torch.zeros(1, 32769, device="cuda")
    with pytest.raises(GdrError) as e:
        layer.norm_forward(big, big[0])
    assert e.value.status == 2
    with pytest.raises(GdrError) as e:
        layer.norm_backward(x, x, w, workspace=torch.empty(1, device="cuda", dtype=torch.uint8))
    assert e.value.status == 5


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,D", [(7, 33), (700, 250), (1300, 887), (1300, 2133), (700, 4089)])
@pytest.mark.parametrize("quant", [None, "row", 32, 128])
def test_a_row_does_not_see_its_neighbours(rows, D, quant, io):
    """Rows that share an aligned vector with their neighbours' ends, which hold NaN and infinity."""
    gen = torch.Generator().manual_seed(rows)
    x, res, dy = (torch.randn(rows, D, generator=gen).to(io).cuda() for _ in range(3))
    w = torch.randn(D, generator=gen).to(io).cuda()
    clean = layer.norm_forward(x, w, res, eps=EPS, quant=quant)
    dx = layer.norm_backward(dy, clean[1], w, eps=EPS)[0]
    bad = torch.arange(rows, device="cuda") % 3 == 1
    x[bad], dy[bad] = float("nan"), float("inf")
    got = layer.norm_forward(x, w, res, eps=EPS, quant=quant)
    for a, b in zip(clean, got):
        if a is not None:
            assert torch.equal(a[~bad].view(torch.uint8), b[~bad].view(torch.uint8))
    assert torch.equal(dx[~bad], layer.norm_backward(dy, got[1], w, eps=EPS)[0][~bad])
    assert got[1][bad].isnan().all() and (quant is None or got[3][bad].isnan().all())


LONG_ODD = [(400, 2553), (400, 5001), (310, 8191), (305, 16001), (305, 32761), (3, 32767), (310, 32767)]


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,D", LONG_ODD)
def test_long_odd_rows(rows, D, io):
    test_forward(rows, D, io)
    test_eight_bits(rows, D, io, "row")
    test_eight_bits(rows, D, io, 64)
    test_backward(rows, D, io, True)


NARROW = [*range(1, 21), 67, 3000]


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", range(1, 10))
def test_rows_narrower_than_a_vector(D, io):
    """Rows of 1 to 9 columns: a vector of 8 spans several of them, and those of more than one row end past the tensor."""
    for rows in NARROW:
        test_forward(rows, D, io)
        test_eight_bits(rows, D, io, "row")
        test_eight_bits(rows, D, io, 32)


@pytest.mark.parametrize("with_dr", [False, True])
@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", range(1, 10))
def test_backward_of_rows_narrower_than_a_vector(D, io, with_dr):
    """From 2433 rows on a block has a next row on its way; the tensors' last vectors hold the ends of several rows.

    dw of a column: at most 2 rows a thread's sum, 76 partial sums in turn and 5 additions of a tree, each within 2^-24 of
    the sum of the terms' sizes, and 4 roundings a term: 87 x 2^-24 = 5.2e-6 of it."""
    for rows in (1, 2, 5, 8, 13, 600, 2432, 2433, 2440, 3001):
        r, dy, w = make(rows, D, io, seed=rows)
        dr = make(rows, D, io, seed=rows + 1)[0] if with_dr else None
        dx, dw = layer.norm_backward(dy, r, w, dr, eps=EPS)
        want, want_dw = backward_reference(dy, r, w, dr)
        rstd = 1 / torch.sqrt((r.double() ** 2).mean(-1, keepdim=True) + EPS)
        top = (rstd * (dy.double() * w.double()).abs()).amax(-1, keepdim=True) + (dr.double().abs() if with_dr else 0)
        assert bool(((dx.double() - want).abs() <= 1e-5 * top + HALF_ULP[io] * want.abs() + 2.0 ** -24).all())
        size = (dy.double() * r.double() * rstd).abs().sum(0)
        assert bool(((dw.double() - want_dw).abs() <= 5.2e-6 * size + 1e-30).all())


@pytest.mark.parametrize("quant", [2 ** 32 + 32, 2 ** 32, 2 ** 33 + 128, 2 ** 31, 2 ** 63 - 1])
def test_groups_beyond_32_bits_are_refused(quant):
    x, res, w = make(4, 256, torch.bfloat16)
    with pytest.raises(GdrError) as e:
        layer.norm_forward(x, w, res, quant=quant)
    assert e.value.status == 9


def test_backward_of_wide_rows_in_half_the_bytes_takes_no_longer():
    """Rows of 4097 to 8192 columns, which no ring holds: loads that wait for one another took 16-bit rows past fp32's time."""
    def fastest(io):
        r, dy, w = make(4096, 8192, io, seed=9)
        times = []
        for _ in range(12):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            layer.norm_backward(dy, r, w, r)
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end))
        return min(times)

    whole = fastest(torch.float32)
    assert fastest(torch.bfloat16) < whole and fastest(torch.float16) < whole
