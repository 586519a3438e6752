"""The gated linear recurrence where its tiles wait for one another: long sequences of few channels, batches whose sequences
take turns, more tiles than blocks.  Tolerances are those of the short ones: with sigmoid decays (0.88 at the middle) a term
lives for tens of tokens, whatever the length.
"""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import gdr, layer
from test_gpu_lru import check, make
from test_gpu_lru_backward import compare, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,D,form", [(1, 5000, 96, "direct"), (3, 2000, 200, "direct"), (5, 1700, 33, "direct"),
                                        (2, 900, 2080, "rate")])
def test_against_64_bits(B, T, D, form, io):
    s = make((B, T), D, io, form)
    dy, dh = randn(B, T, D, io=io, seed=1), randn(B, D, seed=2)
    y, h, kept = layer.lru_forward(**s, want_kept=True)
    got = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], dh, kept)
    for i in range(B):
        check(s, i, i, y, h, io)
    compare(s, range(B), dy, dh, got, io)
    assert gdr.gdr_get_device_status() == 0


@pytest.mark.parametrize("io,pad", [(torch.bfloat16, 0), (torch.bfloat16, 1), (torch.float32, 0), (torch.float32, 3)])
@pytest.mark.parametrize("B,T,D", [(3, 2000, 200), (7, 3000, 64), (40, 130, 520), (300, 9, 72)])
def test_a_batch_is_its_sequences(B, T, D, io, pad):
    """Each sequence by itself has the bits that it has in the batch, and packed."""
    s = make((B, T), D, io, "rate", pad=pad)
    dy = randn(B, T, D, io=io, seed=1)
    y, h, kept = layer.lru_forward(**s, want_kept=True)
    d = layer.lru_backward(s["x"], s["r"], s["i"], s["lam"], dy, s["h0"], kept=kept)
    for i in (0, B // 2, B - 1):
        one = {k: (v if k == "lam" else v[i:i + 1]) for k, v in s.items()}
        y1, h1, _ = layer.lru_forward(**one)
        d1 = layer.lru_backward(one["x"], one["r"], one["i"], one["lam"], dy[i:i + 1], one["h0"])
        assert torch.equal(y1[0], y[i]) and torch.equal(h1[0], h[i])
        for name in ("dx", "dr", "di", "dh0"):
            assert torch.equal(getattr(d1, name)[0], getattr(d, name)[i]), name
    cu = torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
    flat = {k: (v.flatten(0, 1) if k in ("x", "r", "i") else v) for k, v in s.items()}
    y2, h2, _ = layer.lru_forward(**flat, cu_seqlens=cu)
    d2 = layer.lru_backward(flat["x"], flat["r"], flat["i"], flat["lam"], dy.flatten(0, 1), flat["h0"], cu_seqlens=cu)
    assert torch.equal(y2.unflatten(0, (B, T)), y) and torch.equal(h2, h)
    assert torch.equal(d2.dx.unflatten(0, (B, T)), d.dx) and torch.equal(d2.dr.unflatten(0, (B, T)), d.dr)
