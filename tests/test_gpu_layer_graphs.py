"""A decoding step and a training step of the layer operators, captured into CUDA graphs: replays on new inputs give the
bits of eager calls (every sum has a fixed order), and states move on from replay to replay."""
import pytest
import torch

from chunked_gated_delta_prepare_gb300 import layer

pytestmark = pytest.mark.gpu
D, N, H, K, POOL = 192, 16, 2, 64, 6


def randn(*shape, dtype=torch.bfloat16):
    return torch.randn(*shape, device="cuda").to(dtype)


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


def test_decoding_step():
    torch.manual_seed(0)
    slots = torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda")
    w, wc, A = randn(D), randn(D, 4), -torch.rand(D, N, device="cuda")
    x, res = randn(3, D), randn(3, D)
    first = [randn(POOL, 3, D), randn(POOL, D, N, dtype=torch.float32), randn(POOL, H, K, K, dtype=torch.float32)]
    states = [s.clone() for s in first]

    def step(states):
        y, r, _, _ = layer.norm_forward(x, w, res)
        c = layer.conv_step(y, wc, None, states[0], slots=slots)
        bc = c[:, :N].reshape(3, 1, N).contiguous()
        s = layer.ssm_step(c, y, A, bc, bc, states[1], z=r, slots=slots)
        q = c[:, :H * K].reshape(3, H, K).contiguous()
        return s, layer.delta_step(q, q, q, gate, beta, states[2], slots=slots)

    gate, beta = -torch.rand(3, H, device="cuda"), torch.full((3, H), 0.5, device="cuda", dtype=torch.bfloat16)
    graph, out = capture(lambda: step(states))
    for s, f in zip(states, first):
        s.copy_(f)
    eager = [s.clone() for s in first]
    for _ in range(3):
        x.copy_(randn(3, D))
        graph.replay()
        want = step(eager)
        torch.cuda.synchronize()
        for a, b in zip((*out, *states), (*want, *eager)):
            assert torch.equal(a, b)


def test_training_step():
    torch.manual_seed(1)
    B, T = 2, 70
    w, wc, A, bias = randn(D), randn(D, 4), -torch.rand(D, N, device="cuda"), randn(D)
    x, z, dy, bc = randn(B, T, D), randn(B, T, D), randn(B, T, D), randn(B, T, 1, N)

    def step():
        y, r, _, _ = layer.norm_forward(x, w)
        c, _ = layer.conv_forward(y, wc, bias)
        s, _ = layer.ssm_forward(c, y, A, bc, bc, z=z)
        grads = layer.ssm_backward(c, y, A, bc, bc, dy, z=z)
        gc = layer.conv_backward(y, wc, bias, grads.dx)
        gn = layer.norm_backward(gc[0], r, w)
        return s, grads.dA, grads.dB, grads.dC, gc[1], gc[2], *gn

    graph, out = capture(step)
    for _ in range(2):
        x.copy_(randn(B, T, D))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
