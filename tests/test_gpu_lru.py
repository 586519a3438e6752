"""The gated linear recurrence (prompts, packed prompts, single tokens) against the recurrence in 64 bits.

Tolerances.  Every term of a state carries a product of decays.  Each decay is off by at most 2^-21 of itself (the
hardware's 2^x and reciprocal), on average by less than 1e-8 near 1 (measured), beside its own rounding of 2^-25, which
falls to both sides; terms live for up to 1000 tokens here, which leaves 1e-5.  The input's part is off by a few 2^-22.
States and fp32 outputs are held to 2e-5 of the sum of their terms' sizes, 16-bit outputs to half a unit on top.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import GdrError, gdr, layer
from lru_reference import scan

pytestmark = pytest.mark.gpu
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
TOL = 2e-5
FORMS = [("rate", True), ("rate", False), ("direct", True), ("direct", False)]


def make(lead, D, io, form="rate", gate=True, seed=0, n=None, pad=0, h0=True):
    """Inputs of tokens `lead`; pad: x, r and i as slices of wider rows, `pad` elements apart."""
    gen = torch.Generator().manual_seed(seed)

    def wide():
        row = torch.randn(*lead, D + 2 * pad, generator=gen).to(io).cuda()
        return row[..., pad:pad + D]

    s = dict(x=wide(), r=wide(), i=wide() if gate else None, lam=None, h0=None)
    if form == "rate":                 # a channel with its gate open keeps 0.9 to 0.999 of its state a token
        s["lam"] = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(D, generator=gen)) / 8)).cuda()
    else:
        s["r"].add_(2)
    if h0:
        s["h0"] = torch.randn(n or lead[0], D, generator=gen).cuda()
    return s


def part(s, rows):
    return {k: (s[k] if k == "lam" or s[k] is None else s[k][rows]) for k in ("x", "r", "i", "lam")}


def check(s, i, rows, y, h, io, c=8.0):
    """Sequence i, its tokens given by `rows` (an index of the leading dimensions)."""
    hs, sizes = scan(**part(s, rows), h0=None if s["h0"] is None else s["h0"][i], c=c)
    err = (y[rows].double() - hs[1:]).abs()
    assert bool((err <= TOL * sizes[1:] + HALF_ULP[io] * hs[1:].abs() + 2.0 ** -24).all()), (i, float(err.max()))
    if h is not None:
        assert bool(((h[i].double() - hs[-1]).abs() <= TOL * sizes[-1] + 1e-30).all()), i


SHAPES = [(1, 1, 1, 0), (2, 3, 5, 1), (1, 8, 64, 0), (2, 17, 66, 2), (1, 127, 130, 3), (3, 128, 64, 8), (1, 129, 63, 0),
          (2, 300, 72, 1), (1, 1000, 40, 0), (4, 40, 1030, 0), (1, 513, 257, 0)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form,gate", FORMS)
@pytest.mark.parametrize("B,T,D,pad", SHAPES)
def test_batches(B, T, D, pad, form, gate, io):
    s = make((B, T), D, io, form, gate, pad=pad, h0=T % 2 == 1)
    y, h, none = layer.lru_forward(**s)
    assert none is None and gdr.gdr_last_variant() == "lru"
    for i in range(B):
        check(s, i, i, y, h, io)
    y2, none, kept = layer.lru_forward(**s, want_h_final=False, want_kept=True)
    assert none is None and torch.equal(y, y2)
    # the kept states: each in front of 128 tokens
    tiles = -(-T // 128)
    assert kept.shape == (B * tiles, D) and kept.dtype == torch.float32
    hs, sizes = scan(**part(s, B - 1), h0=None if s["h0"] is None else s["h0"][B - 1])
    for k in range(tiles):
        err = (kept[(B - 1) * tiles + k].double() - hs[128 * k]).abs()
        assert bool((err <= TOL * sizes[128 * k] + 1e-30).all())


LENGTHS = [[5], [0], [1, 0, 2, 3], [64, 64], [700, 0, 1, 33, 0], [0, 0, 127, 128, 129], [3] * 70, [0, 256, 0, 1]]


def bounds(lens):
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    at = cu.tolist()
    return cu, [slice(a, b) for a, b in zip(at, at[1:])]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("D,form,gate", [(40, "rate", True), (264, "direct", True), (65, "direct", False), (7, "rate", False)])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, D, form, gate, io):
    s = make((sum(lens),), D, io, form, gate, n=len(lens))
    cu, rows = bounds(lens)
    y, h, _ = layer.lru_forward(**s, cu_seqlens=cu)
    for i, at in enumerate(rows):
        check(s, i, at, y, h, io)
        if at.start == at.stop:
            assert torch.equal(h[i], s["h0"][i])
    s["h0"] = None
    y, h, _ = layer.lru_forward(**s, cu_seqlens=cu)
    for i, at in enumerate(rows):
        check(s, i, at, y, h, io)


def test_a_sequence_does_not_see_its_neighbours():
    lens = [100, 190, 300]
    cu, rows = bounds(lens)
    s = make((590,), 72, torch.float32, n=3)
    y, h, _ = layer.lru_forward(**s, cu_seqlens=cu)
    bad = {k: (v if k == "lam" else v.clone()) for k, v in s.items()}
    for k in ("x", "r", "i"):
        bad[k][:100], bad[k][290:] = float("nan"), float("inf")
    bad["h0"][0] = float("nan")
    y2, h2, _ = layer.lru_forward(**bad, cu_seqlens=cu)
    assert torch.equal(y[rows[1]], y2[rows[1]]) and torch.equal(h[1], h2[1])
    assert bool(y2[rows[0]].isnan().all()) and bool(h2[0].isnan().all())


def test_a_whole_sequence_is_its_parts():
    """A prompt in two calls, the second from the first's state, and its last tokens one by one."""
    s = make((1, 400), 130, torch.float32)
    y, h, _ = layer.lru_forward(**s)
    cut = lambda a, b: {k: (s[k] if k == "lam" else s[k][:, a:b]) for k in ("x", "r", "i", "lam")}  # noqa: E731
    y1, h1, _ = layer.lru_forward(**cut(0, 173), h0=s["h0"])
    y2, h2, _ = layer.lru_forward(**cut(173, 390), h0=h1)
    pool = torch.cat([torch.zeros_like(h2), h2])
    steps = [layer.lru_step(*(v[0, t][None] for v in (s["x"], s["r"], s["i"])), s["lam"], pool,
                            slots=torch.ones(1, dtype=torch.int32, device="cuda")) for t in range(390, 400)]
    got = torch.cat([y1[0], y2[0], *steps])
    top = float(y.abs().max())
    assert float((got - y[0]).abs().max()) <= TOL * top and float((pool[1:] - h).abs().max()) <= TOL * top
    assert not pool[0].any()


def test_gates_at_their_ends():
    """Open and shut gates: the state is kept as it is, or replaced."""
    inf = float("inf")
    for form in ("rate", "direct"):
        s = make((1, 6), 4, torch.float32, form)
        s["r"][0, 2], s["r"][0, 4] = -inf, inf
        s["i"][0, 3], s["i"][0, 5] = -inf, inf
        y, h, _ = layer.lru_forward(**s)
        check(s, 0, 0, y, h, torch.float32)
        if form == "rate":               # a shut recurrence gate keeps the state and takes nothing
            assert torch.equal(y[0, 2], y[0, 1])
        else:                            # an open forget gate keeps it, a shut one takes the input alone
            assert torch.equal(y[0, 4], y[0, 3])
    # rates that keep everything, or nothing
    s = make((1, 300), 4, torch.float32)
    s["lam"] = torch.tensor([-200.0, -30.0, 20.0, 200.0], device="cuda")
    y, h, _ = layer.lru_forward(**s)
    check(s, 0, 0, y, h, torch.float32)
    assert torch.equal(y[0, :, 0], s["h0"][0, :1].expand(300))


def test_nan_stays_in_its_channel_and_after_its_token():
    for form in ("rate", "direct"):
        for key in ("x", "r", "i"):
            s = make((1, 300), 70, torch.bfloat16, form)
            clean, _, _ = layer.lru_forward(**s)
            s[key][0, 140, 11] = float("nan")
            y, h, _ = layer.lru_forward(**s)
            assert bool(y[0, 140:, 11].isnan().all()) and bool(h[0, 11].isnan())
            y[0, 140:, 11] = clean[0, 140:, 11]
            assert torch.equal(y, clean)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form,gate", FORMS)
@pytest.mark.parametrize("n,D,pad", [(1, 1, 0), (3, 65, 1), (16, 1000, 8), (70, 4098, 0)])
def test_step(n, D, pad, form, gate, io):
    s = make((n,), D, io, form, gate, pad=pad, h0=False)
    gen = torch.Generator().manual_seed(9)
    h = torch.randn(n + 5, D, generator=gen).cuda()
    slots = torch.randperm(n + 5, generator=gen)[:n].to(torch.int32).cuda()
    if n > 2:
        slots[1], slots[2] = -1, n + 5                   # two padding rows
        s["x"][1], s["r"][2] = float("nan"), float("inf")
    first = h.clone()
    y = layer.lru_step(s["x"], s["r"], s["i"], s["lam"], h, slots=slots)
    used = torch.zeros(n + 5, dtype=torch.bool)
    for row, slot in enumerate(slots.tolist()):
        if not 0 <= slot < n + 5:
            assert not y[row].any()
            continue
        used[slot] = True
        one = {k: (s[k] if k == "lam" or s[k] is None else s[k][row][None]) for k in ("x", "r", "i", "lam")}
        hs, sizes = scan(**one, h0=first[slot])
        assert bool(((h[slot].double() - hs[1]).abs() <= 4e-6 * sizes[1] + 1e-30).all())
        assert bool(((y[row].double() - hs[1]).abs() <= 4e-6 * sizes[1] + HALF_ULP[io] * hs[1].abs() + 2.0 ** -24).all())
    assert torch.equal(h[~used.cuda()], first[~used.cuda()])
    # without slots, row i uses state i
    h, again = first.clone(), first.clone()
    if n > 2:
        s["x"][1], s["r"][2] = 0, 0
    y = layer.lru_step(s["x"], s["r"], s["i"], s["lam"], h)
    z = layer.lru_step(s["x"], s["r"], s["i"], s["lam"], again, slots=torch.arange(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, z) and torch.equal(h, again) and torch.equal(h[n:], first[n:])


def test_the_rate_constant():
    s = make((1, 50), 8, torch.float32)
    y, h, _ = layer.lru_forward(**s, c=1.5)
    check(s, 0, 0, y, h, torch.float32, c=1.5)


def test_same_bits_again_and_on_another_stream():
    s = make((5000,), 600, torch.bfloat16, n=3)
    cu, _ = bounds([4000, 0, 1000])
    want = layer.lru_forward(**s, cu_seqlens=cu, want_kept=True)[:2]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, layer.lru_forward(**s, cu_seqlens=cu)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer.lru_forward(**s, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_beyond_32_bits():
    T, D = 530_000, 4100                                  # 2.17e9 elements a tensor
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, r = (torch.randn(1, T, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y, h, kept = layer.lru_forward(x, r, want_kept=True)
    at = T // 128 * 128 - 256
    y2, h2, _ = layer.lru_forward(x[:, at:], r[:, at:], h0=kept[at // 128][None])
    assert torch.equal(y[:, at:], y2) and torch.equal(h, h2)
    hs, sizes = scan(x[0, at:], r[0, at:], h0=kept[at // 128])
    assert bool(((h2[0].double() - hs[-1]).abs() <= TOL * sizes[-1]).all())


def test_refusals():
    s = make((2, 5), 8, torch.bfloat16)
    cu = torch.tensor([0, 3, 10], dtype=torch.int32, device="cuda")
    flat = {k: (v.flatten(0, 1) if k in ("x", "r", "i") else v) for k, v in s.items()}
    for base, bad in ((s, dict(r=None)), (s, dict(r=s["r"][:1])), (s, dict(i=s["i"].float())), (s, dict(lam=s["lam"][:4])),
                      (s, dict(lam=s["lam"].double())), (s, dict(h0=s["h0"][:1])), (s, dict(x=s["x"].double())),
                      (s, dict(x=s["x"].cpu())), (s, dict(x=s["x"][0])), (flat, dict(cu_seqlens=cu.long())),
                      (flat, dict(cu_seqlens=cu[:1])), (s, dict(cu_seqlens=cu)),
                      (s, dict(x=s["x"][:, :0], r=s["r"][:, :0], i=s["i"][:, :0]))):
        with pytest.raises(ValueError):
            layer.lru_forward(**(base | bad))
    for kw, status in ((dict(c=0.0), 9), (dict(c=float("nan")), 9), (dict(c=float("inf")), 9)):
        with pytest.raises(GdrError) as e:
            layer.lru_forward(**s, **kw)
        assert e.value.status == status
    layer.lru_forward(**(s | dict(lam=None)), c=0.0)       # not used
    long = make((1, 500), 8, torch.bfloat16)
    with pytest.raises(GdrError) as e:
        layer.lru_forward(**long, workspace=torch.empty(16, device="cuda"))
    assert e.value.status == 5
    x, h = torch.zeros(3, 8, device="cuda"), torch.zeros(2, 8, device="cuda")
    with pytest.raises(GdrError) as e:                     # more rows than states
        layer.lru_step(x, x, None, None, h)
    assert e.value.status == 2
    for bad in (dict(h=h[:, :4]), dict(h=h.half()), dict(slots=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(x=x[None])):
        with pytest.raises(ValueError):
            layer.lru_step(**(dict(x=x, r=x, i=None, lam=None, h=h) | bad))
