"""Workloads of the operators of a recurrent layer with input and forget gates: the gated linear recurrence (prompts, training,
single tokens), the layer norm in front of its projections, and the gated norm of a recurrence's output.

`run` computes one pass in plain torch operations (`own` false) or through the library (`own` true) on what `prepare`
made; `exact` computes the same in 64 bits, token by token; `work` counts what a pass has to move and compute.

Shapes: T tokens (a batch of B equal sequences, or `seqs` packed ones), D channels, H heads of V columns.
The recurrence: h_t = a_t h_{t-1} + u_t with
    form "rate":    log a = -c softplus(lam) sigmoid(r),  u = sqrt(1 - a^2) sigmoid(i) x     (lam: a rate for each channel)
    form "direct":  a = sigmoid(r),                       u = (1 - a) sigmoid(i) x           (without i: (1 - a) x)
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ES = {"bf16": 2, "f16": 2, "f32": 4}
LN_EPS, GN_EPS, RATE = 1e-5, 1e-6, 8.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token of 16 sequences through the recurrence, the states in a pool: latency
        dict(name="lru_step_16", op="lru_step", B=16, D=4096, form="rate", gate=True, io="bf16"),
        # one token of 256 sequences, a gate without rates and without an input gate
        dict(name="lru_step_256", op="lru_step", B=256, D=8192, form="direct", gate=False, io="f16"),
        # one long prompt: few channels for the GPU, many tokens
        dict(name="lru_prompt_32k", op="lru_prompt", T=32768, seqs=1, D=4096, form="rate", gate=True, io="bf16"),
        # nine ragged prompts packed (one empty), fp32 throughout, an odd number of channels
        dict(name="lru_ragged_5k", op="lru_prompt", T=5003, seqs=9, D=1001, form="direct", gate=True, io="f32"),
        # a training step of 4 x 2048 tokens with every gradient
        dict(name="lru_train_4x2k", op="lru_train", B=4, T=2048, D=4096, form="rate", gate=True, io="bf16"),
        # the norm before the projections of one decoding step: 16 sequences, latency
        dict(name="ln_step_16", op="ln", rows=16, D=4096, io="bf16"),
        # the same norm over a 32k-token prompt
        dict(name="ln_prompt_32k", op="ln", rows=32768, D=4096, io="bf16"),
        # forward and backward of the norm in a training step of 4 x 2048 tokens
        dict(name="ln_train_8k", op="ln_train", rows=8192, D=2048, io="bf16"),
        # the same in fp32 with rows that are no multiple of a vector
        dict(name="ln_train_odd", op="ln_train", rows=4451, D=2278, io="f32"),
        # the output norm of one token of 64 sequences, 32 heads of 128
        dict(name="gnorm_step_64", op="gnorm", T=64, H=32, V=128, act="silu", per_head=False, io="bf16"),
        # the output norm of a 32k-token prompt
        dict(name="gnorm_prompt_32k", op="gnorm", T=32768, H=32, V=128, act="silu", per_head=False, io="bf16"),
        # a training step of 4 x 2048 tokens, 16 heads of 128, a sigmoid gate and weights of each head
        dict(name="gnorm_train_8k", op="gnorm_train", T=8192, H=16, V=128, act="sigmoid", per_head=True, io="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges; its main tensors hold no more bytes than the largest listed case's of its kind."""
    op = rng.choice(["lru_step", "lru_prompt", "lru_train", "ln", "ln_train", "gnorm", "gnorm_train"])
    c = dict(op=op, io=rng.choice(["bf16", "bf16", "f16", "f32"]))
    most = 2 ** (26 if op.endswith("train") else 28) // ES[c["io"]]           # values of one tensor
    if op in ("ln", "ln_train"):
        c["D"] = _log(rng, 64, 8192)
        c["rows"] = _log(rng, 1, min(32768, most // c["D"]))
        return c
    if op in ("gnorm", "gnorm_train"):
        c["V"], c["H"] = rng.choice([64, 128, 128, 256, _log(rng, 16, 1024)]), _log(rng, 1, 64)
        c["T"] = _log(rng, 1, min(32768, most // (c["V"] * c["H"])))
        c["act"], c["per_head"] = rng.choice(["silu", "sigmoid"]), rng.random() < 0.5
        return c
    c["form"], c["gate"] = rng.choice(["rate", "direct"]), rng.random() < 0.7
    c["D"] = _log(rng, 64, 8192)
    if op == "lru_step":
        c["B"] = _log(rng, 1, 256)
    elif op == "lru_prompt":
        c["T"] = _log(rng, 1, min(32768, most // c["D"]))
        c["seqs"] = rng.randint(1, min(16, c["T"]))
    else:
        c["B"] = rng.randint(1, 4)
        c["T"] = _log(rng, 1, min(8192, most // (c["D"] * c["B"])))
    return c


def lengths(case):
    """The lengths of the packed sequences: uneven, the second of four or more empty."""
    n, T = case["seqs"], case["T"]
    rng = random.Random(n * 1000003 + T)
    share = [rng.uniform(0.1, 1.0) ** 2 for _ in range(n)]
    if n >= 4:
        share[1] = 0.0
    lens = [int(T * s / sum(share)) for s in share]
    lens[-1] += T - sum(lens)
    return lens


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, io = case["op"], DT[case["io"]]

    def randn(*shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype or io)

    s = dict(case=case, op=op)
    if op in ("ln", "ln_train"):
        rows, D = case["rows"], case["D"]
        # the residual stream: rows with a mean of their own
        s["x"] = randn(rows, D, scale=0.5)
        s["res"] = (2 * torch.randn(rows, D, generator=gen, device="cuda") +
                    torch.randn(rows, 1, generator=gen, device="cuda")).to(io)
        s["w"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(io)
        s["b"] = randn(D, scale=0.1)
        if op == "ln_train":
            s["dy"], s["dr"] = randn(rows, D), randn(rows, D, scale=0.3)
        return s
    if op in ("gnorm", "gnorm_train"):
        T, H, V = case["T"], case["H"], case["V"]
        s["x"] = randn(T, H, V, scale=0.1)
        # the gate is a slice of the layer's input projection, its queries, keys or values beside it
        s["z"] = randn(T, H * V + -(-H * V // 16) * 8)[:, :H * V].unflatten(1, (H, V))
        s["w"] = (1 + 0.1 * torch.randn(*((H, V) if case["per_head"] else (V,)), generator=gen, device="cuda")).to(io)
        if op == "gnorm_train":
            s["dy"] = randn(T, H, V)
        return s
    D = case["D"]
    lead = (case["B"], case["T"]) if op == "lru_train" else (case["T"],) if op == "lru_prompt" else (case["B"],)
    s["x"] = randn(*lead, D)
    gates = randn(*lead, 2 * -(-D // 8) * 8)               # one projection gives r and i
    s["r"] = gates[..., :D]
    s["i"] = gates[..., gates.shape[-1] // 2:][..., :D] if case["gate"] else None
    s["lam"] = None
    if case["form"] == "rate":
        # a channel with its gate open keeps 0.9 to 0.999 of its state a token
        keep = -torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda")) / RATE
        s["lam"] = torch.log(torch.expm1(keep))
    else:
        s["r"].add_(2)                                      # forget gates start open
    if op == "lru_step":
        S = case["B"] + 8
        slots = torch.randperm(S - 1, generator=gen, device="cuda")[:case["B"]].to(torch.int32)
        if case["B"] >= 9:
            slots[case["B"] // 2] = -1                     # a padding row
        s["slots"], s["h"] = slots, randn(S, D, dtype=torch.float32)
    elif op == "lru_prompt":
        s["h"] = randn(case["seqs"], D, dtype=torch.float32)
        s["cu"] = torch.tensor([0] + lengths(case)).cumsum(0).to(torch.int32).cuda()
    else:
        s["dy"] = randn(*lead, D)
    return s


# ---------------------------------------------------------------- plain forms (32 bits, rounded once at the end)

def _plain_ln(s):
    io = s["x"].dtype
    s32 = s["x"].float() + s["res"].float()
    mid = s32 - s32.mean(-1, keepdim=True)
    y = mid * torch.rsqrt((mid * mid).mean(-1, keepdim=True) + LN_EPS) * s["w"].float() + s["b"].float()
    return dict(y=y.to(io), r=s32.to(io))


def _plain_ln_train(s):
    out, io = _plain_ln(s), s["x"].dtype
    r, dy = out["r"].float(), s["dy"].float()              # the backward reads r as it was kept
    mid = r - r.mean(-1, keepdim=True)
    rstd = torch.rsqrt((mid * mid).mean(-1, keepdim=True) + LN_EPS)
    xh, wdy = mid * rstd, dy * s["w"].float()
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True)) + s["dr"].float()
    return dict(**out, dx=dx.to(io), dw=(dy * xh).sum(0), db=dy.sum(0))


def _gate(z, act):
    """The gate's value and slope."""
    sig = torch.sigmoid(z)
    return (z * sig, sig * (1 + z * (1 - sig))) if act == "silu" else (sig, sig * (1 - sig))


def _plain_gnorm(s):
    x, (f, _) = s["x"].float(), _gate(s["z"].float(), s["case"]["act"])
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + GN_EPS)
    return dict(y=(n * s["w"].float() * f).to(s["x"].dtype))


def _plain_gnorm_train(s):
    io, x, w, dy = s["x"].dtype, s["x"].float(), s["w"].float(), s["dy"].float()
    f, slope = _gate(s["z"].float(), s["case"]["act"])
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + GN_EPS)
    n, dn = x * rstd, dy * w * f
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    dw = (dy * n * f).sum(0)
    return dict(y=(n * w * f).to(io), dx=dx.to(io), dz=(dy * n * w * slope).to(io),
                dw=dw if s["case"]["per_head"] else dw.sum(0))


def _plain_gates(s):
    """The decay, 1 - its part (sqrt(1 - a^2) or 1 - a), the input's gate (or 1) and sigmoid(r)."""
    r = s["r"].float()
    sr = torch.sigmoid(r)
    g = torch.sigmoid(s["i"].float()) if s["i"] is not None else torch.ones((), device=r.device)
    if s["lam"] is None:
        return sr, torch.sigmoid(-r), g, sr
    log_a = -RATE * torch.nn.functional.softplus(s["lam"]) * sr
    return torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)), g, sr


def _scan(a, b, dim):
    """h_t = a_t h_{t-1} + b_t along `dim`, from zero: doubles the reach in each step (in place)."""
    T, reach = a.shape[dim], 1
    while reach < T:
        late, early = (lambda v: v.narrow(dim, reach, T - reach)), (lambda v: v.narrow(dim, 0, T - reach))
        late(b).add_(late(a) * early(b))
        late(a).copy_(late(a) * early(a))
        reach *= 2
    return b


def _plain_lru_prompt(s):
    cu, T = s["cu"].long(), s["x"].shape[0]
    a, part, g, _ = _plain_gates(s)
    seq = torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True) - 1
    first = (torch.arange(T, device="cuda") == cu[seq])[:, None]
    b = part * g * s["x"].float()
    b += torch.where(first, a * s["h"][seq], 0)
    h = _scan(a.masked_fill(first, 0.0), b, 0)
    some = (cu[1:] > cu[:-1])[:, None]
    return dict(y=h.to(s["x"].dtype), h=torch.where(some, h[(cu[1:] - 1).clamp_min(0)], s["h"]))


def _plain_lru_train(s):
    io, x = s["x"].dtype, s["x"].float()
    a, part, g, sr = _plain_gates(s)
    h = _scan(a.clone(), part * g * x, 1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)                   # a_{t+1}
    e = _scan(after.flip(1), s["dy"].float().flip(1), 1).flip(1)
    out = dict(y=h.to(io), h=h[:, -1], dx=(e * part * g).to(io))
    if s["i"] is not None:
        out["di"] = (e * part * x * g * (1 - g)).to(io)
    if s["lam"] is None:
        out["dr"] = (e * (before - g * x) * a * part).to(io)
    else:
        dlog = e * a * (before - g * x * a / part)
        out["dr"] = (dlog * (-RATE * torch.nn.functional.softplus(s["lam"])) * sr * (1 - sr)).to(io)
        out["dlam"] = (dlog * sr).sum((0, 1)) * (-RATE * torch.sigmoid(s["lam"]))
    return out


def _plain_lru_step(s):
    ok = (s["slots"] >= 0)[:, None]
    at = torch.where(s["slots"] < 0, s["h"].shape[0] - 1, s["slots"]).long()       # the last slot is nobody's
    old = s["h"][at]
    a, part, g, _ = _plain_gates(s)
    h = a * old + part * g * s["x"].float()
    s["h"][at] = torch.where(ok, h, old)
    return dict(y=torch.where(ok, h, 0).to(s["x"].dtype), h=s["h"])


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from chunked_gated_delta_prepare_gb300 import layer
    op = s["op"]
    if op in ("ln", "ln_train"):
        y, r = layer.layernorm_forward(s["x"], s["w"], s["b"], s["res"], eps=LN_EPS)
        if op == "ln":
            return dict(y=y, r=r)
        dx, dw, db = layer.layernorm_backward(s["dy"], r, s["w"], s["dr"], eps=LN_EPS)
        return dict(y=y, r=r, dx=dx, dw=dw, db=db)
    if op in ("gnorm", "gnorm_train"):
        act = s["case"]["act"]
        y = layer.gated_norm_forward(s["x"], s["z"], s["w"], gate=act, eps=GN_EPS)
        if op == "gnorm":
            return dict(y=y)
        dx, dz, dw = layer.gated_norm_backward(s["dy"], s["x"], s["z"], s["w"], gate=act, eps=GN_EPS)
        return dict(y=y, dx=dx, dz=dz, dw=dw)
    four = (s["x"], s["r"], s["i"], s["lam"])
    if op == "lru_step":
        return dict(y=layer.lru_step(*four, s["h"], c=RATE, slots=s["slots"]), h=s["h"])
    if op == "lru_prompt":
        y, h, _ = layer.lru_forward(*four, s["h"], c=RATE, cu_seqlens=s["cu"])
        return dict(y=y, h=h)
    y, h, kept = layer.lru_forward(*four, c=RATE, want_kept=True)
    d = layer.lru_backward(*four, s["dy"], kept=kept, c=RATE)
    out = dict(y=y, h=h, dx=d.dx, dr=d.dr)
    if s["i"] is not None:
        out["di"] = d.di
    if s["lam"] is not None:
        out["dlam"] = d.dlam
    return out


PLAIN = dict(ln=_plain_ln, ln_train=_plain_ln_train, gnorm=_plain_gnorm, gnorm_train=_plain_gnorm_train,
             lru_step=_plain_lru_step, lru_prompt=_plain_lru_prompt, lru_train=_plain_lru_train)


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass has to move and compute

def work(case):
    op, e = case["op"], ES[case["io"]]
    if op in ("ln", "ln_train"):
        n, D = case["rows"] * case["D"], case["D"]
        if op == "ln":                                  # x, res, y, r
            return dict(bytes=4 * n * e + 2 * D * e, flops=10 * n)
        return dict(bytes=8 * n * e + D * (3 * e + 8), flops=26 * n)               # and r, dy, dr, dx
    if op in ("gnorm", "gnorm_train"):
        n = case["T"] * case["H"] * case["V"]
        w = case["V"] * (case["H"] if case["per_head"] else 1)
        if op == "gnorm":                               # x, z, y
            return dict(bytes=3 * n * e + w * e, flops=10 * n)
        return dict(bytes=8 * n * e + w * (2 * e + 4), flops=32 * n)               # and dy, x, z, dx, dz
    D, gates = case["D"], 2 if case["gate"] else 1
    lam = 4 * D if case["form"] == "rate" else 0
    if op == "lru_step":
        n = case["B"] * D
        return dict(bytes=(2 + gates) * n * e + 8 * n + lam, flops=25 * n)
    if op == "lru_prompt":
        n = case["T"] * D
        return dict(bytes=(2 + gates) * n * e + 8 * case["seqs"] * D + lam, flops=25 * n)
    n = case["B"] * case["T"] * D                       # x, r, i, y; x, r, i, dy, dx, dr, di
    return dict(bytes=(5 + 3 * gates) * n * e + 4 * case["B"] * D + 3 * lam, flops=75 * n)


# ---------------------------------------------------------------- the definition in 64 bits

def _sig64(x):
    return 1 / (1 + torch.exp(-x))


def _exact_ln(s, case):
    x = s["x"].double() + s["res"].double()
    r = x.to(s["x"].dtype).double()
    w, b = s["w"].double(), s["b"].double()
    dev = torch.sqrt(x.var(1, unbiased=False) + LN_EPS)[:, None]
    out = dict(y=(x - x.mean(1)[:, None]) / dev * w + b, r=r)
    if case["op"] == "ln":
        return out
    dev = torch.sqrt(r.var(1, unbiased=False) + LN_EPS)[:, None]
    c, dy, D = r - r.mean(1)[:, None], s["dy"].double(), r.shape[1]
    t = dy * w
    # the derivative of (r_j - m) / dev by r_k is ((j = k) - 1 / D) / dev - c_j c_k / (D dev^3)
    dx = t / dev - t.sum(1)[:, None] / (D * dev) - c * (t * c).sum(1)[:, None] / (D * dev ** 3) + s["dr"].double()
    return dict(**out, dx=dx, dw=(dy * c / dev).sum(0), db=dy.sum(0))


def _exact_gnorm(s, case):
    x, z, w = s["x"].double(), s["z"].double(), s["w"].double()
    size = torch.sqrt(x.pow(2).sum(2) / x.shape[2] + GN_EPS)[..., None]
    sig = _sig64(z)
    f = z * sig if case["act"] == "silu" else sig
    out = dict(y=x / size * w * f)
    if case["op"] == "gnorm":
        return out
    slope = sig + z * sig * _sig64(-z) if case["act"] == "silu" else sig * _sig64(-z)
    dy = s["dy"].double()
    t = dy * w * f
    out["dx"] = t / size - x * (t * x).sum(2)[..., None] / (x.shape[2] * size ** 3)
    out["dz"] = dy * x / size * w * slope
    dw = torch.einsum("thv,thv->hv", dy, x / size * f)
    out["dw"] = dw if case["per_head"] else torch.einsum("hv->v", dw)
    return out


def _exact_lru(s, case):
    x, r = s["x"].double(), s["r"].double()
    q = _sig64(r)
    g = _sig64(s["i"].double()) if s["i"] is not None else torch.ones_like(x)
    if case["form"] == "rate":
        lam = s["lam"].double()
        k = RATE * (torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs())))
        a = torch.exp(-k * q)
        part = torch.sqrt(-torch.expm1(-2 * k * q))
    else:
        a, part = q, _sig64(-r)
    u = part * g * x
    op = case["op"]
    if op == "lru_step":
        y, h = torch.zeros_like(x), s["h"].double()
        for j, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                h[slot] = a[j] * h[slot] + u[j]
                y[j] = h[slot]
        return dict(y=y, h=h)
    if op == "lru_prompt":
        y, last, at = torch.empty_like(x), [], 0
        for j, n in enumerate(lengths(case)):
            h = s["h"][j].double()
            for t in range(at, at + n):
                h = torch.addcmul(u[t], a[t], h, out=y[t])
            last.append(h)
            at += n
        return dict(y=y, h=torch.stack(last))
    T = x.shape[1]
    hs = torch.zeros(x.shape[0], T + 1, x.shape[2], device=x.device, dtype=x.dtype)
    for t in range(T):
        hs[:, t + 1] = a[:, t] * hs[:, t] + u[:, t]
    e, run_e = torch.empty_like(x), torch.zeros_like(x[:, 0])
    for t in range(T - 1, -1, -1):
        e[:, t] = run_e + s["dy"][:, t].double()
        run_e = e[:, t] * a[:, t]
    out = dict(y=hs[:, 1:], h=hs[:, -1], dx=e * part * g)
    if s["i"] is not None:
        out["di"] = e * part * x * g * _sig64(-s["i"].double())
    if case["form"] == "rate":
        # by log a: of a itself a, of sqrt(1 - a^2) -a^2 / sqrt(1 - a^2)
        dlog = e * (a * hs[:, :-1] - a * a / part * g * x)
        out["dr"] = -dlog * k * q * _sig64(-r)
        out["dlam"] = -(dlog * q).sum(1).sum(0) * RATE * _sig64(lam)
    else:
        out["dr"] = e * (hs[:, :-1] - g * x) * q * _sig64(-r)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("ln"):
        return _exact_ln(s, case)
    if op.startswith("gnorm"):
        return _exact_gnorm(s, case)
    return _exact_lru(s, case)
