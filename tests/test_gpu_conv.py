"""The short causal convolution (prompts, packed prompts, gradient, single tokens) against its definition in 64 bits.

Tolerances.  A preactivation is five fp32 operations on exact inputs, silu a handful more with relative error below
1e-6: fp32 outputs are held to 1e-5 of the sum of the absolute terms, 16-bit outputs to half a unit in their last place
on top.  Sums over tokens (dw, db) are held to 1e-5 of the sum of their terms' sizes.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, layer

pytestmark = pytest.mark.gpu
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def randn(*shape, io=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(io).cuda()


def one(x, w, b, state, silu):
    """One sequence in 64 bits: y, the state it leaves, and the size of the terms."""
    W = w.shape[1]
    state = torch.zeros(W - 1, x.shape[1], device="cuda", dtype=torch.double) if state is None else state.double()
    rows = torch.cat([state, x.double()])
    win = rows.unfold(0, W, 1) if x.shape[0] else rows.new_zeros(0, x.shape[1], W)
    pre = (win * w.double()).sum(-1) + (b.double() if b is not None else 0)
    size = (win * w.double()).abs().sum(-1) + (b.double().abs() if b is not None else 0)
    return (pre * torch.sigmoid(pre) if silu else pre), rows[x.shape[0]:], size


def check_sequences(xs, ys, outs, w, b, states, silu, io):
    for i, x in enumerate(xs):
        want, state, size = one(x, w, b, states[i] if states is not None else None, silu)
        assert bool(((ys[i].double() - want).abs() <= 1e-5 * size + HALF_ULP[io] * want.abs() + 2.0 ** -24).all()), i
        if outs is not None:
            assert torch.equal(outs[i].double(), state), i


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("B,T,D,W,silu,bias,with_state", [
    (1, 1, 1, 4, True, True, True), (2, 2, 8, 4, True, False, False), (3, 3, 7, 2, False, True, True),
    (2, 17, 64, 3, True, True, True), (1, 100, 250, 4, True, True, False), (2, 513, 256, 4, True, True, True),
    (1, 130, 2050, 4, False, False, True), (2, 64, 520, 2, True, True, False), (1, 4097, 33, 3, True, False, True)])
def test_batches(B, T, D, W, silu, bias, with_state, io):
    x, w = randn(B, T, D, io=io), randn(D, W, io=io, seed=1)
    b = randn(D, io=io, seed=2) if bias else None
    state = randn(B, W - 1, D, io=io, seed=3) if with_state else None
    y, out = layer.conv_forward(x, w, b, state, silu=silu)
    check_sequences(x, y, out, w, b, state, silu, io)
    y2, none = layer.conv_forward(x, w, b, state, silu=silu, want_state=False)
    assert none is None and torch.equal(y, y2)


LENGTHS = [[5], [0], [1, 0, 2, 3], [64, 64], [700, 0, 1, 33, 0], [0, 0, 127, 128, 129], [3] * 70]


def packed(lens, D, W, io, ld=None, seed=0):
    total, n = sum(lens), len(lens)
    x = randn(total, ld or D, io=io, seed=seed)[:, :D]
    state = randn(n, W - 1, D, io=io, seed=seed + 1)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    return x, state, cu


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("D,ld", [(40, 40), (264, 1000), (65, 67)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, D, ld, io):
    x, state, cu = packed(lens, D, 4, io, ld)
    w, b = randn(D, 4, io=io, seed=5), randn(D, io=io, seed=6)
    y, out = layer.conv_forward(x, w, b, state, cu_seqlens=cu)
    check_sequences(x.split(lens), y.split(lens), out, w, b, state, True, io)
    y, out = layer.conv_forward(x, w, b, cu_seqlens=cu)
    check_sequences(x.split(lens), y.split(lens), out, w, b, None, True, io)


def test_a_sequence_does_not_see_its_neighbours():
    lens = [40, 30, 50]
    x, state, cu = packed(lens, 64, 4, torch.float32)
    w = randn(64, 4, seed=5)
    y, out = layer.conv_forward(x, w, None, state, cu_seqlens=cu)
    bad = x.clone()
    bad[:40], bad[70:] = float("nan"), float("inf")
    z, zout = layer.conv_forward(bad, w, None, state, cu_seqlens=cu)
    assert torch.equal(y[40:70], z[40:70]) and torch.equal(out[1], zout[1])
    dy = randn(120, 64, seed=6)
    dx = layer.conv_backward(x, w, None, dy, state, cu_seqlens=cu)[0]
    dy[:40], dy[70:] = float("nan"), float("inf")
    assert torch.equal(dx[40:70], layer.conv_backward(bad, w, None, dy, state, cu_seqlens=cu)[0][40:70])


def backward_check(xs, dys, w, b, states, d_outs, silu, io, got):
    dx, dw, db, dstate = got
    W = w.shape[1]
    want_w, size_w = torch.zeros_like(w, dtype=torch.double), torch.zeros_like(w, dtype=torch.double)
    want_b, size_b = want_w[:, 0].clone(), want_w[:, 0].clone()
    at = 0
    for i, (x, dy) in enumerate(zip(xs, dys)):
        n = x.shape[0]
        state = states[i].double() if states is not None else torch.zeros(W - 1, x.shape[1], device="cuda",
                                                                           dtype=torch.double)
        rows = torch.cat([state, x.double()])
        drows, size = torch.zeros_like(rows), torch.zeros_like(rows)
        if n:
            win = rows.unfold(0, W, 1)
            pre = (win * w.double()).sum(-1) + (b.double() if b is not None else 0)
            sig = torch.sigmoid(pre)
            dp = dy.double() * (sig * (1 + pre * (1 - sig)) if silu else 1)
            # dp has the preactivation's rounding, so its own error is relative to the size of dy
            big = dy.double().abs() * (1.1 + (win * w.double()).abs().sum(-1) * 0.5 if silu else 1)
            for j in range(W):
                drows[j:j + n] += w.double()[:, j] * dp
                size[j:j + n] += (w.double()[:, j]).abs() * big
                want_w[:, j] += (dp * rows[j:j + n]).sum(0)
                size_w[:, j] += (big * rows[j:j + n].abs()).sum(0)
            want_b += dp.sum(0)
            size_b += big.sum(0)
        if d_outs is not None:
            drows[n:] += d_outs[i].double()
            size[n:] += d_outs[i].double().abs()
        ok = (drows.abs() * HALF_ULP[io] + 1e-5 * size + 2.0 ** -24)
        assert bool(((dx[at:at + n].double() - drows[W - 1:]).abs() <= ok[W - 1:]).all()), i
        if states is not None:
            assert bool(((dstate[i].double() - drows[:W - 1]).abs() <= ok[:W - 1]).all()), i
        at += n
    assert bool(((dw.double() - want_w).abs() <= 1e-5 * size_w + 1e-30).all())
    if b is not None:
        assert bool(((db.double() - want_b).abs() <= 1e-5 * size_b + 1e-30).all())
    else:
        assert db is None


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("B,T,D,W,silu,bias,with_state", [
    (1, 1, 1, 4, True, True, True), (2, 2, 8, 4, True, False, True), (3, 3, 7, 2, False, True, True),
    (2, 33, 64, 3, True, True, True), (1, 100, 250, 4, True, True, False), (2, 513, 132, 4, True, True, True),
    (1, 130, 2050, 4, False, False, False), (4, 300, 68, 2, True, True, False)])
def test_backward(B, T, D, W, silu, bias, with_state, io):
    x, w, dy = randn(B, T, D, io=io), randn(D, W, io=io, seed=1), randn(B, T, D, io=io, seed=4)
    b = randn(D, io=io, seed=2) if bias else None
    state = randn(B, W - 1, D, io=io, seed=3) if with_state else None
    d_out = randn(B, W - 1, D, io=io, seed=5) if with_state else None
    got = layer.conv_backward(x, w, b, dy, state, d_out, silu=silu)
    backward_check(x, dy, w, b, state, d_out, silu, io, (got[0].flatten(0, 1), *got[1:]))
    again = layer.conv_backward(x, w, b, dy, state, d_out, silu=silu)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,ld", [(40, 40), (264, 1000), (65, 67)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_backward_packed(lens, D, ld, io):
    x, state, cu = packed(lens, D, 4, io, ld)
    w, b, dy = randn(D, 4, io=io, seed=5), randn(D, io=io, seed=6), randn(sum(lens), D, io=io, seed=7)
    d_out = randn(len(lens), 3, D, io=io, seed=8)
    got = layer.conv_backward(x, w, b, dy, state, d_out, cu_seqlens=cu)
    backward_check(x.split(lens), dy.split(lens), w, b, state, d_out, True, io, got)


def test_backward_against_differences():
    x, w, b, state = randn(1, 6, 3), randn(3, 4, seed=1), randn(3, seed=2), randn(1, 3, 3, seed=3)
    dy, d_out = randn(1, 6, 3, seed=4), randn(1, 3, 3, seed=5)
    got = layer.conv_backward(x, w, b, dy, state, d_out)

    def loss(args):
        y, left, _ = one(args[0][0], args[1], args[2], args[3][0], True)
        return float((y * dy[0].double()).sum() + (left * d_out[0].double()).sum())

    base, h = [t.double() for t in (x, w, b, state)], 1e-5
    for k in range(4):
        for i in range(0, base[k].numel(), 2):
            hi, lo = ([t.clone() for t in base] for _ in range(2))
            hi[k].view(-1)[i] += h
            lo[k].view(-1)[i] -= h
            assert float(got[k].reshape(-1)[i]) == pytest.approx((loss(hi) - loss(lo)) / (2 * h), rel=1e-4, abs=1e-4)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("n,D,W,silu,ld", [(1, 1, 4, True, 1), (3, 7, 2, False, 9), (2, 64, 3, True, 64),
                                           (70, 1032, 4, True, 2064), (5, 250, 4, True, 250)])
def test_step(n, D, W, silu, ld, io):
    pool = n + 5
    w, b = randn(D, W, io=io, seed=1), randn(D, io=io, seed=2)
    state = randn(pool, W - 1, D, io=io, seed=3)
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32).cuda()
    x = randn(n, ld, io=io, seed=4)[:, :D]
    pad = []
    if n > 2:
        pad = [0, n - 1]
        slots[0], slots[n - 1] = -1, pool
        x = x.clone() if ld == D else x
        x[0] = float("nan")
    before = state.clone()
    y = layer.conv_step(x, w, b, state, silu=silu, slots=slots)
    for i in range(n):
        if i in pad:
            assert not y[i].any()
            continue
        s = int(slots[i])
        check_sequences([x[i:i + 1]], [y[i:i + 1]], [state[s]], w, b, [before[s]], silu, io)
        before[s] = state[s]
    assert torch.equal(before, state)         # no other state moved
    z = layer.conv_step(x[:1], w, b, state[:1].clone(), silu=silu)
    if n <= 2:
        check_sequences([x[:1]], [z], None, w, b, state[:1], silu, io)


def test_steps_go_on_from_a_prompt():
    x, w, b = randn(2, 20, 96, io=torch.bfloat16), randn(96, 4, io=torch.bfloat16, seed=1), None
    whole, last = layer.conv_forward(x, w, b)
    _, state = layer.conv_forward(x[:, :12], w, b)
    for t in range(12, 20):
        assert torch.equal(layer.conv_step(x[:, t], w, b, state), whole[:, t])
    assert torch.equal(state, last)


def test_another_stream():
    side = torch.cuda.Stream()
    x, w, dy = randn(2, 3000, 512), randn(512, 4, seed=1), randn(2, 3000, 512, seed=2)
    side.wait_stream(torch.cuda.current_stream())
    y, _ = layer.conv_forward(x, w, stream=side)
    got = layer.conv_backward(x, w, None, dy, stream=side)
    side.synchronize()
    assert torch.equal(y, layer.conv_forward(x, w)[0])
    assert torch.equal(got[1], layer.conv_backward(x, w, None, dy)[1])


def test_refusals():
    x, w, state = randn(2, 5, 8), randn(8, 4, seed=1), randn(2, 3, 8, seed=2)
    cu = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    for call in (lambda: layer.conv_forward(x[0], w), lambda: layer.conv_forward(x, w, cu_seqlens=cu),
                 lambda: layer.conv_forward(x.flatten(0, 1), w, cu_seqlens=cu.long()),
                 lambda: layer.conv_forward(x, w[:4]), lambda: layer.conv_forward(x, w.bfloat16()),
                 lambda: layer.conv_forward(x, w, state=state[:1]), lambda: layer.conv_forward(x[:, :0], w),
                 lambda: layer.conv_forward(x.cpu(), w), lambda: layer.conv_forward(x.double(), w.double()),
                 lambda: layer.conv_backward(x, w, None, x[:1]), lambda: layer.conv_step(x, w, None, state),
                 lambda: layer.conv_step(x[0], w, None, state.transpose(0, 1)),
                 lambda: layer.conv_step(x[0], w, None, state, slots=torch.zeros(5, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: layer.conv_forward(x, randn(8, 5)), 2), (lambda: layer.conv_forward(x, randn(8, 1)), 2),
                         (lambda: layer.conv_step(x[0], w, None, state), 2),        # 5 rows, 2 states
                         (lambda: layer.conv_backward(x, w, None, x, workspace=torch.empty(8, device="cuda")), 5)):
        with pytest.raises(GdrError) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [2500, 2501, 2502])
def test_long_runs(D, io):
    """Enough tokens and channels for the longest runs, whole and cut short by the sequences' ends."""
    lens = [3000, 129, 0, 2500, 64, 2307]
    x, state, cu = packed(lens, D, 4, io)
    w, b = randn(D, 4, io=io, seed=5), randn(D, io=io, seed=6)
    y, out = layer.conv_forward(x, w, b, state, cu_seqlens=cu)
    check_sequences(x.split(lens), y.split(lens), out, w, b, state, True, io)
    dy, d_out = randn(sum(lens), D, io=io, seed=7), randn(len(lens), 3, D, io=io, seed=8)
    got = layer.conv_backward(x, w, b, dy, state, d_out, cu_seqlens=cu)
    backward_check(x.split(lens), dy.split(lens), w, b, state, d_out, True, io, got)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("D", [33, 65, 130])
def test_a_row_does_not_see_its_neighbours(D, io):
    """Rows that share an aligned word or vector with their neighbours' ends, which hold NaN and infinity."""
    lens = [40, 30, 50]
    x, state, cu = packed(lens, D, 4, io)
    w, dy = randn(D, 4, io=io, seed=5), randn(120, D, io=io, seed=6)
    y = layer.conv_forward(x, w, None, state, cu_seqlens=cu)[0]
    dx = layer.conv_backward(x, w, None, dy, state, cu_seqlens=cu)[0]
    x[:40], x[70:], dy[:40], dy[70:] = float("nan"), float("inf"), float("inf"), float("nan")
    assert torch.equal(y[40:70], layer.conv_forward(x, w, None, state, cu_seqlens=cu)[0][40:70])
    assert torch.equal(dx[40:70], layer.conv_backward(x, w, None, dy, state, cu_seqlens=cu)[0][40:70])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("D", [5, 64, 131])
def test_tensors_that_start_at_one_element(D, io):
    """x is a slice from column 1 on, dy and the states start one element into their memory."""
    B, T = 2, 37

    def shifted(*shape, seed):
        t = randn(*shape, io=io, seed=seed)
        out = torch.empty(t.numel() + 1, dtype=io, device="cuda")[1:].view(shape)
        return out.copy_(t)

    x = randn(B, T, D + 3, io=io)[..., 1:D + 1]
    w, b = shifted(D, 4, seed=1), shifted(D, seed=2)
    state, dy = shifted(B, 3, D, seed=3), shifted(B, T, D, seed=4)
    y, out = layer.conv_forward(x, w, b, state)
    check_sequences(x, y, out, w, b, state, True, io)
    got = layer.conv_backward(x, w, b, dy, state)
    backward_check(x, dy, w, b, state, None, True, io, (got[0].flatten(0, 1), *got[1:]))


def test_taps_beyond_32_bits_are_refused():
    w = torch.empty(1, 2 ** 32 + 4, dtype=torch.bfloat16, device="cuda")       # 8.6 GB that nobody reads
    x = torch.zeros(1, 8, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(GdrError) as e:
        layer.conv_forward(x, w, want_state=False)
    assert e.value.status == 2
    del w
    torch.cuda.empty_cache()
