"""The gated linear recurrence, the layer norm and the gated norm together, as a layer runs them: a decoding step and a
training step against 64 bits, captured into CUDA graphs, and on two streams at once."""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import gdr, layer
from lru_reference import scan, scan_backward

pytestmark = pytest.mark.gpu
H, V, POOL = 3, 32, 7
D = H * V


def randn(*shape, io=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, device="cuda")).to(io)


def weights(io):
    torch.manual_seed(0)
    return dict(w=1 + randn(D, io=io, scale=0.1), b=randn(D, io=io, scale=0.1), inp=randn(4 * D, D, io=io, scale=D ** -0.5),
                lam=torch.rand(D, device="cuda") * 2 - 5, g=1 + randn(V, io=io, scale=0.1))


def forward(p, x, res, cu=None, states=None, slots=None, **kw):
    """norm -> projection -> recurrence -> gated norm.  With states: one token of each row."""
    y, r = layer.layernorm_forward(x, p["w"], p["b"], res)
    z = y @ p["inp"].t()
    a, i, u, gate = (z[..., k * D:(k + 1) * D] for k in range(4))
    if states is not None:
        h, kept = layer.lru_step(u, a, i, p["lam"], states, slots=slots), None
    else:
        h, last, kept = layer.lru_forward(u, a, i, p["lam"], cu_seqlens=cu, want_kept=True)
        kw["last"] = last
    o = layer.gated_norm_forward(h.unflatten(-1, (H, V)), gate.unflatten(-1, (H, V)), p["g"])
    return o, r, dict(y=y, u=u, a=a, i=i, gate=gate, h=h, kept=kept, **kw)


def test_decoding_goes_on_from_packed_prompts():
    """The last tokens one by one from the states that the prompts left, in other slots of a pool, a padding row between."""
    io = torch.float32
    p, lens, steps = weights(io), [37, 1, 300], 3
    x, res = randn(sum(lens) + 3 * steps, D, io=io), randn(sum(lens) + 3 * steps, D, io=io)
    whole = torch.tensor([0] + [n + steps for n in lens]).cumsum(0).to(torch.int32).cuda()
    want, r, _ = forward(p, x, res, whole)
    rows = [torch.arange(a, a + n) for a, n in zip(whole.tolist(), lens)]
    head = torch.cat(rows).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    _, _, mid = forward(p, x[head], res[head], cu)
    states = torch.full((POOL, D), 7.0, device="cuda")
    slots = torch.tensor([5, -1, 2, 3], dtype=torch.int32, device="cuda")
    states[slots[[0, 2, 3]].long()] = mid["last"]
    for k in range(steps):
        at = torch.tensor([whole[j] + lens[j] + k for j in range(3)], device="cuda")
        rows = torch.stack([at[0], at[0], at[1], at[2]])
        got, _, _ = forward(p, x[rows], res[rows], states=states, slots=slots)
        # fp32 all through; the same sums in other orders
        assert float((got[[0, 2, 3]] - want[at]).abs().max()) <= 1e-4 * float(want.abs().max())
        assert not got[1].any()
    assert bool((states[[0, 1, 4, 6]] == 7.0).all())


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_training_step_against_64_bits(io):
    """The layer's gradients chained by hand, against the same chain of the definitions in 64 bits on the same inputs."""
    p = weights(io)
    x, res = randn(2, 150, D, io=io), randn(2, 150, D, io=io)
    o, r, s = forward(p, x, res)
    do = randn(2, 150, H, V, io=io)
    heads = lambda t: t.unflatten(-1, (H, V))  # noqa: E731
    dh, dgate, dg = layer.gated_norm_backward(do, heads(s["h"]), heads(s["gate"]), p["g"])
    d = layer.lru_backward(s["u"], s["a"], s["i"], p["lam"], dh.flatten(2), kept=s["kept"])
    dz = torch.cat([d.dr, d.di, d.dx, dgate.flatten(2)], -1)
    dy = dz @ p["inp"]
    dx, dw, db = layer.layernorm_backward(dy, r, p["w"])

    # each operator against its definition, on the inputs that it was given: 16 bits round in between
    tol = {torch.float32: 3e-5, torch.bfloat16: 2.0 ** -8 + 3e-5}[io]

    def near(got, want, tol=tol):
        assert float((got.double() - want).abs().max()) <= tol * float(want.abs().max())

    def norm(t, q):
        t = t.double()
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * q["g"].double()

    h64, z64, g64 = (t.double().requires_grad_() for t in (heads(s["h"]), heads(s["gate"]), p["g"]))
    want = norm(h64, dict(g=g64)) * z64 * torch.sigmoid(z64)
    near(o, want.detach())
    for got, grad in zip((dh, dgate, dg), torch.autograd.grad(want, (h64, z64, g64), do.double())):
        near(got, grad)
    total = 0
    for k in range(2):
        hs, _ = scan(s["u"][k], s["a"][k], s["i"][k], p["lam"])
        near(s["h"][k], hs[1:])
        ref = scan_backward(s["u"][k], s["a"][k], s["i"][k], p["lam"], dh.flatten(2)[k])
        near(d.dx[k], ref["dx"][0])
        near(d.dr[k], ref["dr"][0])
        near(d.di[k], ref["di"][0])
        total = total + ref["dlam"][0]
    near(d.dlam, total, 1e-4)
    s64, w64, b64 = r.double().requires_grad_(), p["w"].double().requires_grad_(), p["b"].double().requires_grad_()
    want = torch.nn.functional.layer_norm(s64, (D,), w64, b64, 1e-5)
    for got, grad in zip((dx, dw, db), torch.autograd.grad(want, (s64, w64, b64), dy.double())):
        near(got, grad)


def capture(f):
    """f run once as a warm-up and once into a graph, on a side stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


def test_decoding_step_in_a_graph():
    io = torch.bfloat16
    p, x, res = weights(io), randn(3, D, io=io), randn(3, D, io=io)
    slots = torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda")
    first = randn(POOL, D)
    states, eager = first.clone(), first.clone()
    graph, (o, r, _) = capture(lambda: forward(p, x, res, states=states, slots=slots))
    states.copy_(first)
    for _ in range(3):
        x.copy_(randn(3, D, io=io))
        graph.replay()
        want, want_r, _ = forward(p, x, res, states=eager, slots=slots)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(r, want_r) and torch.equal(states, eager)


def training(p, x, do):
    o, r, s = forward(p, x, x)
    heads = lambda t: t.unflatten(-1, (H, V))  # noqa: E731
    dh, dgate, dg = layer.gated_norm_backward(do, heads(s["h"]), heads(s["gate"]), p["g"])
    d = layer.lru_backward(s["u"], s["a"], s["i"], p["lam"], dh.flatten(2), kept=s["kept"])
    again = layer.lru_backward(s["u"], s["a"], s["i"], p["lam"], dh.flatten(2))
    return o, r, dh, dgate, dg, *d[:4], *again[:4], *layer.layernorm_backward(d.dx, r, p["w"])


@pytest.mark.parametrize("B,T", [(2, 70), (2, 1000)])
def test_training_step_in_graphs(B, T):
    """Two graphs of the same step, replayed in turn; each replay gives the bits of eager calls on its inputs."""
    io = torch.bfloat16
    p = weights(io)
    x, do = randn(B, T, D, io=io), randn(B, T, H, V, io=io)
    graphs = [capture(lambda: training(p, x, do)) for _ in range(2)]
    for k in range(4):
        x.copy_(randn(B, T, D, io=io))
        graph, out = graphs[k % 2]
        graph.replay()
        want = training(p, x, do)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    """Long scans, whose blocks wait for one another, on two streams at the same time."""
    io = torch.bfloat16
    p = weights(io)
    work = [(randn(1, 20_000, D, io=io), randn(1, 20_000, H, V, io=io)) for _ in range(2)]
    want = [training(p, *w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for _ in range(3):
        got = []
        for w, s in zip(work, streams):
            with torch.cuda.stream(s):
                got.append(training(p, *w))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert gdr.gdr_get_device_status() == 0                 # no wait gave up


def test_a_workspace_of_the_callers_own():
    """One workspace for calls one after another, larger than any of them needs and full of anything."""
    x, r = randn(1, 700, D), randn(1, 700, D)
    dy = randn(1, 700, D)
    ws = torch.full((1 << 22,), 0xA5, device="cuda", dtype=torch.uint8)
    want = layer.lru_forward(x, r)[0]
    grads = layer.lru_backward(x, r, None, None, dy)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        assert torch.equal(layer.lru_forward(x, r, workspace=ws)[0], want)
        again = layer.lru_backward(x, r, None, None, dy, workspace=ws)
        assert torch.equal(again.dx, grads.dx) and torch.equal(again.dr, grads.dr)
        n = layer.layernorm_backward(dy, x, r[0, 0].contiguous(), workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(n, layer.layernorm_backward(dy, x, r[0, 0].contiguous())))
        h = [t.unflatten(-1, (H, V)) for t in (dy, x, r)]
        g = layer.gated_norm_backward(*h, r[0, 0, :V].contiguous(), workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(g, layer.gated_norm_backward(*h, r[0, 0, :V].contiguous())))


def test_autograd_beside_captured_gradients():
    """A captured gradient while an eager graph of the same leaves is alive."""
    io = torch.float32
    x, r = randn(1, 300, D, io=io).requires_grad_(), randn(1, 300, D, io=io).requires_grad_()

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, r):
            y, _, kept = layer.lru_forward(x, r, want_kept=True)
            ctx.save_for_backward(x, r, kept)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, r, kept = ctx.saved_tensors
            d = layer.lru_backward(x, r, None, None, dy, kept=kept)
            return d.dx, d.dr

    eager = Scan.apply(x, r)                                # its graph lives on
    dy = randn(1, 300, D, io=io)
    graph, out = capture(lambda: layer.lru_backward(x.detach(), r.detach(), None, None, dy)[:2])
    graph.replay()
    torch.cuda.synchronize()
    want = torch.autograd.grad(eager, (x, r), dy)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


FAR, WIDE = 1_060_000, 2048                                 # more than 2^31 values


def test_recurrence_past_2_31_values():
    """A short sequence behind a very long one: the bits of the short one alone."""
    io, tail = torch.bfloat16, 300
    x, r, i, dy = (torch.randn(FAR, WIDE, device="cuda", dtype=io) for _ in range(4))
    lam = torch.rand(WIDE, device="cuda") * 2 - 5
    cu = torch.tensor([0, FAR - tail, FAR], dtype=torch.int32, device="cuda")
    y, h, kept = layer.lru_forward(x, r, i, lam, cu_seqlens=cu, want_kept=True)
    d = layer.lru_backward(x, r, i, lam, dy, kept=kept, cu_seqlens=cu)
    part = [t[-tail:].unsqueeze(0).clone() for t in (x, r, i)]
    want, want_h, _ = layer.lru_forward(*part, lam)
    grads = layer.lru_backward(*part, lam, dy[-tail:].unsqueeze(0).clone())
    assert torch.equal(y[-tail:], want[0]) and torch.equal(h[1], want_h[0])
    for a, b in zip(d[:3], grads[:3]):
        assert torch.equal(a[-tail:], b[0])
    assert gdr.gdr_get_device_status() == 0


def test_norms_past_2_31_values():
    """Their last rows against the definitions; the gradients of the weights with nothing but the last rows in them."""
    io, tail = torch.bfloat16, 8
    x = torch.randn(FAR, WIDE, device="cuda", dtype=io)
    z = torch.randn(FAR, WIDE, device="cuda", dtype=io)
    w = (1 + 0.1 * torch.randn(WIDE, device="cuda")).to(io)
    dy = torch.zeros(FAR, WIDE, device="cuda", dtype=io)
    dy[-tail:] = torch.randn(tail, WIDE, device="cuda").to(io)
    tol = 2.0 ** -8 + 3e-5

    def near(got, want, tol=tol):
        assert float((got.double() - want).abs().max()) <= tol * float(want.abs().max())

    y, s = layer.layernorm_forward(x, w, None, z)
    dx, dw, db = layer.layernorm_backward(dy, s, w)
    s64, w64 = s[-tail:].double().requires_grad_(), w.double().requires_grad_()
    want = torch.nn.functional.layer_norm(s64, (WIDE,), w64, None, 1e-5)
    near(s[-tail:], x[-tail:].double() + z[-tail:].double())
    near(y[-tail:], want.detach(), 2 * tol)                 # of s itself, here of its rounding
    ds, dw64 = torch.autograd.grad(want, (s64, w64), dy[-tail:].double())
    near(dx[-tail:], ds)
    near(dw, dw64, 1e-4)
    near(db, dy[-tail:].double().sum(0), 1e-4)
    del y, s, dx
    heads = lambda t: t.unflatten(-1, (16, WIDE // 16))  # noqa: E731
    g = w[:WIDE // 16].contiguous()
    y = layer.gated_norm_forward(heads(x), heads(z), g)
    dx, dz, dg = layer.gated_norm_backward(heads(dy), heads(x), heads(z), g)
    x64, z64, g64 = (t.double().requires_grad_() for t in (heads(x[-tail:]), heads(z[-tail:]), g))
    want = x64 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + 1e-6) * g64 * z64 * torch.sigmoid(z64)
    near(y[-tail:], want.detach())
    for got, grad in zip((dx[-tail:], dz[-tail:], dg), torch.autograd.grad(want, (x64, z64, g64), heads(dy[-tail:]).double())):
        near(got, grad)
