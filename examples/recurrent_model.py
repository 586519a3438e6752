"""A small language model of recurrent layers on libgdr: packed prompts, single-token decoding from a pool of states,
and training steps.

    python examples/recurrent_model.py

Each layer is  residual + norm -> input projection -> short convolution -> recurrence -> output projection, the
recurrence being the gated delta rule or the selective state space scan.  Serving takes the norm's 8-bit output: a
row's scale commutes with the projection, so it is applied to the product (in bf16 here: torch's product widens the
values first, so the 8 bits save no time in this example).  Decoding continues from the states the
prompt left, and its logits are those of the whole sequence run as a prompt.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunked_gated_delta_prepare_gb300 import gdr, layer  # noqa: E402

VOCAB, DIM, HEADS, HEAD, INNER, STATES, RANK, TAPS = 97, 256, 2, 64, 384, 16, 16, 4
IO = torch.bfloat16


# ---------------------------------------------------------------- gradients for autograd

class Norm(torch.autograd.Function):
    """(y, r) of the norm with the residual's addition."""
    @staticmethod
    def forward(ctx, x, weight, residual):
        y, r, _, _ = layer.norm_forward(x, weight, residual)
        ctx.save_for_backward(r, weight)
        return y, r

    @staticmethod
    def backward(ctx, dy, dr):
        r, weight = ctx.saved_tensors
        dx, dw = layer.norm_backward(dy, r, weight, dr)
        return dx, dw.to(weight.dtype), dx


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return layer.conv_forward(x, weight, bias, want_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        dx, dw, db, _ = layer.conv_backward(x, weight, bias, dy)
        return dx, dw.to(weight.dtype), db.to(bias.dtype)


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, *inputs):                    # q, k, v, g, beta
        inputs = [t.contiguous() for t in inputs]
        ctx.save_for_backward(*inputs)
        return gdr.forward(*inputs, want_h_final=False)[0]

    @staticmethod
    def backward(ctx, do):
        return gdr.backward(*ctx.saved_tensors, None, do.contiguous())[:5]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias):
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias)
        return layer.ssm_forward(x, dt, A, B, C, D, z, dt_bias, want_h_final=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, dt, A, B, C, D, z, dt_bias = ctx.saved_tensors
        d = layer.ssm_backward(x, dt, A, B, C, dy, D, z, dt_bias)
        return d.dx, d.ddt, d.dA, d.dB, d.dC, d.dD, d.dz, d.ddt_bias


# ---------------------------------------------------------------- layers

class Layer:
    """One recurrent layer's weights; `kind` is "delta" or "ssm"."""

    def __init__(self, kind, gen):
        def weight(*shape, scale=None):
            scale = shape[-1] ** -0.5 if scale is None else scale
            return (torch.randn(*shape, generator=gen) * scale).to(IO).cuda()

        self.kind = kind
        self.norm = torch.ones(DIM, dtype=IO, device="cuda")
        if kind == "delta":
            self.channels = 3 * HEADS * HEAD
            self.inp = weight(self.channels + 2 * HEADS, DIM)          # q, k, v, then the gate's and beta's logits
            self.out = weight(DIM, HEADS * HEAD)
        else:
            self.channels = INNER
            self.inp = weight(2 * INNER, DIM)                          # x, z
            self.bc = weight(RANK + 2 * STATES, INNER)                 # dt's low rank, B, C
            self.dt = weight(INNER, RANK)
            self.A = -torch.arange(1, STATES + 1, dtype=torch.float32, device="cuda").repeat(INNER, 1)
            self.D = torch.ones(INNER, device="cuda")
            self.dt_bias = torch.full((INNER,), -3.0, device="cuda")
            self.out = weight(DIM, INNER)
        self.taps, self.bias = weight(self.channels, TAPS, scale=0.5), weight(self.channels, scale=0.1)

    def parameters(self):
        return [t for t in vars(self).values() if isinstance(t, torch.Tensor)]

    def new_states(self, slots):
        conv = torch.zeros(slots, TAPS - 1, self.channels, dtype=IO, device="cuda")
        shape = (HEADS, HEAD, HEAD) if self.kind == "delta" else (INNER, STATES)
        return conv, torch.zeros(slots, *shape, device="cuda")

    def delta_inputs(self, conv, logits):
        q, k, v = (t.unflatten(-1, (HEADS, HEAD)) for t in conv.split(HEADS * HEAD, -1))
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(IO) for t in (q, k))
        gate, beta = logits.split(HEADS, -1)
        return q, k, v, torch.nn.functional.logsigmoid(gate.float()) / 16, torch.sigmoid(beta)

    def scan_inputs(self, x, z):
        """The scan's arguments: dt, B and C are projections of x."""
        low, B, C = (x @ self.bc.t()).split([RANK, STATES, STATES], -1)
        return (x, low @ self.dt.t(), self.A, B.unsqueeze(-2), C.unsqueeze(-2)), (self.D, z, self.dt_bias)

    def serve(self, x, residual, states, cu=None, slots=None):
        """Packed prompts [total, DIM] (cu), whose final states go to the pool's slots, or one token of each row."""
        _, r, x8, scale = layer.norm_forward(x, self.norm, residual, quant="row", want_y=False)
        p = ((x8.to(IO) @ self.inp.t()).float() * scale).to(IO)
        conv_states, pool = states
        c = p[:, :self.channels]
        if cu is not None:
            c, left = layer.conv_forward(c, self.taps, self.bias, cu_seqlens=cu)
            conv_states[slots.long()] = left
        else:
            c = layer.conv_step(c, self.taps, self.bias, conv_states, slots=slots)
        rest = p[:, self.channels:]
        if self.kind == "delta":
            q, k, v, g, beta = (t.contiguous() for t in self.delta_inputs(c, rest))
            if cu is not None:
                o, h = gdr.forward_varlen(q, k, v, g, beta, cu)
                pool[slots.long()] = h
            else:
                o = layer.delta_step(q, k, v, g, beta, pool, slots=slots)
        else:
            first, more = self.scan_inputs(c, rest)
            if cu is not None:
                o, h = layer.ssm_forward(*first, *more, cu_seqlens=cu)
                pool[slots.long()] = h
            else:
                o = layer.ssm_step(*first, pool, *more, slots=slots)
        return o.flatten(1) @ self.out.t(), r

    def train(self, x, residual):
        """x, residual [B, T, DIM] -> the layer's output and the new residual."""
        y, r = Norm.apply(x, self.norm, residual)
        p = y @ self.inp.t()
        c = Conv.apply(p[..., :self.channels], self.taps, self.bias)
        rest = p[..., self.channels:]
        if self.kind == "delta":
            o = Delta.apply(*self.delta_inputs(c, rest))
        else:
            (x, dt, A, B, C), (D, z, dt_bias) = self.scan_inputs(c, rest)
            o = Scan.apply(x, dt, A, B, C, D, z, dt_bias)
        return o.flatten(2) @ self.out.t(), r


class Model:
    def __init__(self, kinds=("delta", "ssm"), seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.embed = (torch.randn(VOCAB, DIM, generator=gen) * DIM ** -0.5).to(IO).cuda()
        self.layers = [Layer(kind, gen) for kind in kinds]
        self.norm = torch.ones(DIM, dtype=IO, device="cuda")

    def parameters(self):
        return [self.embed, self.norm] + [p for one in self.layers for p in one.parameters()]

    def new_states(self, slots):
        return [one.new_states(slots) for one in self.layers]

    def serve(self, tokens, states, slots, cu=None):
        """Logits of every token.  tokens [total] packed prompts (cu), or [n] one token of each row."""
        r = self.embed[tokens]
        x = torch.zeros_like(r)
        for one, s in zip(self.layers, states):
            x, r = one.serve(x, r, s, cu, slots)
        return layer.norm_forward(x, self.norm, r)[0] @ self.embed.t()

    def loss(self, tokens):
        """Next-token loss of tokens [B, T + 1]."""
        r = self.embed[tokens[:, :-1]]
        x = torch.zeros_like(r)
        for one in self.layers:
            x, r = one.train(x, r)
        logits = Norm.apply(x, self.norm, r)[0] @ self.embed.t()
        return torch.nn.functional.cross_entropy(logits.float().flatten(0, 1), tokens[:, 1:].flatten())


def decode_gap(model, lengths=(37, 5, 64), steps=6, seed=1):
    """Prompts of these lengths, then `steps` tokens one by one: the largest difference of their logits from those of
    the whole sequences run as prompts, and the largest logit."""
    gen = torch.Generator().manual_seed(seed)
    whole = [torch.randint(VOCAB, (n + steps,), generator=gen).cuda() for n in lengths]
    n = len(lengths)

    def packed(parts):
        cu = torch.tensor([0] + [len(t) for t in parts]).cumsum(0).to(torch.int32).cuda()
        return torch.cat(parts), cu

    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    tokens, cu = packed(whole)
    want = model.serve(tokens, model.new_states(n), slots, cu).split([len(t) for t in whole])
    # decoding: the sequences sit in other slots of a larger pool, a padding row between them
    slots = torch.arange(n + 2, 2, -1, dtype=torch.int32, device="cuda")
    states = model.new_states(n + 3)
    tokens, cu = packed([t[:-steps] for t in whole])
    model.serve(tokens, states, slots, cu)
    rows = torch.cat([slots[:1], torch.full((1,), -1, dtype=torch.int32, device="cuda"), slots[1:]])
    gap = 0.0
    for k in range(steps):
        token = torch.stack([t[len(t) - steps + k] for t in whole])
        logits = model.serve(torch.cat([token[:1], token[:1], token[1:]]), states, rows)
        for i, got in enumerate(torch.cat([logits[:1], logits[2:]])):
            gap = max(gap, float((got.float() - want[i][len(whole[i]) - steps + k].float()).abs().max()))
    return gap, float(torch.cat(want).float().abs().max())


def train(model, steps=20, lr=0.05, seed=2):
    """Losses of plain gradient steps on a repeated batch."""
    gen = torch.Generator().manual_seed(seed)
    tokens = torch.randint(VOCAB, (2, 129), generator=gen).cuda()
    params = model.parameters()
    master = [p.float() for p in params]
    losses = []
    for p in params:
        p.requires_grad_(True)
    for _ in range(steps):
        loss = model.loss(tokens)
        grads = torch.autograd.grad(loss, params)
        losses.append(float(loss.detach()))
        size = torch.stack([g.float().square().sum() for g in grads]).sum().sqrt()
        with torch.no_grad():
            for p, m, g in zip(params, master, grads):
                m -= lr * g.float() / size.clamp_min(1.0)
                p.copy_(m)
    return losses


def main():
    model = Model()
    gap, top = decode_gap(model)
    print(f"decoding against the whole prompt: logits differ by at most {gap:.3f} of {top:.1f}")
    losses = train(model)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
