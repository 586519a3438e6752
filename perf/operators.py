"""Workloads of the operators around the recurrence of a layer: the root-mean-square norm with the residual's
addition and an 8-bit output, the short causal convolution, the selective state space scan and the gated delta
rule's single-token step.

`run` computes one pass in plain torch operations (`own` false) or through the library (`own` true) on what
`prepare` made; `exact` computes the same in 64 bits, token by token; `work` counts what a pass has to move and
compute.

Shapes: T tokens (a batch of B equal sequences, or `seqs` packed ones), D channels, N states a channel, G groups
of channels that share B and C, W convolution taps, H query/key heads and HV value heads of 128 x 128 states.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
TAPS = 4


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the norm before the projections of one decoding step: 16 sequences, 8-bit input of the product, latency
        dict(name="norm8_step_16", op="norm8", rows=16, D=4096, group=0, io="bf16"),
        # the same norm over a 32k-token prompt, a scale for each 128 columns
        dict(name="norm8_prompt_32k", op="norm8", rows=32768, D=4096, group=128, io="bf16"),
        # forward and backward of the norm in a training step of 4 x 2048 tokens
        dict(name="norm_train_8k", op="norm_train", rows=8192, D=2048, io="bf16"),
        # q, k and v of 32 heads of 128 through the convolution: 11 packed prompts, one of them empty
        dict(name="conv_prompt_16k", op="conv_prompt", T=16384, seqs=11, D=12288, io="bf16"),
        # the convolution of 16 heads' q, k and v in a training step, with its gradients
        dict(name="conv_train_4x2k", op="conv_train", B=4, T=2048, D=6144, io="bf16"),
        # one token of 64 sequences through the convolution, the states in a pool
        dict(name="conv_step_64", op="conv_step", B=64, D=6144, io="bf16"),
        # one token of 64 sequences through the selective scan, the states in a pool
        dict(name="ssm_step_64", op="ssm_step", B=64, D=4096, N=16, G=1, io="bf16"),
        # one long prompt: few channels for the GPU, many tokens
        dict(name="ssm_prompt_32k", op="ssm_prompt", T=32768, seqs=1, D=4096, N=16, G=1, io="bf16"),
        # nine ragged prompts packed (one empty), fp32 throughout, a number of states that is no power of two
        dict(name="ssm_ragged_5k", op="ssm_prompt", T=5003, seqs=9, D=1000, N=12, G=2, io="f32"),
        # a training step of 4 x 2048 tokens with every gradient
        dict(name="ssm_train_4x2k", op="ssm_train", B=4, T=2048, D=2048, N=16, G=1, io="bf16"),
        # the gated delta rule for one token of one sequence of 32 heads: latency
        dict(name="delta_step_1", op="delta_step", B=1, H=32, HV=32, per_k=False, io="bf16"),
        # one token of 128 sequences, 32 value heads on 16 query/key heads, a gate for each key dimension
        dict(name="delta_step_128", op="delta_step", B=128, H=16, HV=32, per_k=True, io="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges; its main tensors hold no more than the largest listed case's."""
    op = rng.choice(["norm8", "norm_train", "conv_prompt", "conv_train", "conv_step", "ssm_step", "ssm_prompt",
                     "ssm_train", "delta_step"])
    c = dict(op=op, io=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op in ("norm8", "norm_train"):
        c["D"] = _log(rng, 64, 8192)
        c["rows"] = _log(rng, 1, min(32768, 2 ** 26 // c["D"]))
        if op == "norm8":
            c["group"] = rng.choice([0, 32, 64, 128])
    elif op in ("conv_step", "ssm_step"):
        c["B"], c["D"] = _log(rng, 1, 256), _log(rng, 64, 8192)
        if op == "ssm_step":
            c["G"] = rng.choice([1, 1, 2, 4])
            c["D"], c["N"] = -(-c["D"] // c["G"]) * c["G"], rng.choice([8, 12, 16, 16, 32, 64])
    elif op == "conv_prompt":
        c["D"] = _log(rng, 64, 12288)
        c["T"] = _log(rng, 1, min(32768, 2 ** 27 // c["D"]))
        c["seqs"] = rng.randint(1, min(16, c["T"]))
    elif op == "conv_train":
        c["D"], c["B"] = _log(rng, 64, 8192), rng.randint(1, 4)
        c["T"] = _log(rng, 1, min(8192, 2 ** 26 // (c["D"] * c["B"])))
    elif op == "delta_step":
        c["H"], c["per_k"] = rng.choice([2, 4, 8, 16]), rng.random() < 0.5
        c["HV"], c["B"] = c["H"] * rng.choice([1, 2]), _log(rng, 1, 128)
    else:
        train = op == "ssm_train"
        c["G"], c["N"] = rng.choice([1, 1, 2, 4]), rng.choice([8, 12, 16, 16, 32, 64])
        c["D"] = -(-_log(rng, 64, 4096) // c["G"]) * c["G"]
        most = (2 ** 28 if train else 2 ** 30) // (c["D"] * c["N"])
        if train:
            c["B"] = rng.randint(1, 4)
            c["T"] = _log(rng, 1, min(8192, most // c["B"]))
        else:
            c["T"] = _log(rng, 1, min(32768, most))
            c["seqs"] = rng.randint(1, min(16, c["T"]))
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

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def pool(B):
        """Slots of B sequences in a pool with room; of nine or more, one row is padding (-1). The last slot is free."""
        S = B + 8
        slots = torch.randperm(S - 1, generator=gen, device="cuda")[:B].to(torch.int32)
        if B >= 9:
            slots[B // 2] = -1
        return S, slots

    s = dict(case=case, op=op)
    if op in ("norm8", "norm_train"):
        rows, D = case["rows"], case["D"]
        s["x"], s["res"] = randn(rows, D, scale=0.5), randn(rows, D, scale=2.0)
        s["w"] = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(io)
        if op == "norm_train":
            s["dy"], s["dr"] = randn(rows, D), randn(rows, D, scale=0.3)
        return s
    D = case.get("D")
    if op.startswith("conv"):
        s["w"], s["b"] = randn(D, TAPS, scale=0.5), randn(D, scale=0.1)
        if op == "conv_step":
            S, s["slots"] = pool(case["B"])
            s["x"], s["state"] = randn(case["B"], D), randn(S, TAPS - 1, D)
        elif op == "conv_prompt":
            # the convolution's channels are a slice of the layer's input projection, a gate of D // 3 (q, k, v) beside
            s["x"] = randn(case["T"], D + -(-D // 24) * 8)[:, :D]
            s["state"] = randn(case["seqs"], TAPS - 1, D)
        else:
            s["x"], s["dy"] = randn(case["B"], case["T"], D), randn(case["B"], case["T"], D)
    elif op.startswith("ssm"):
        N, G = case["N"], case["G"]
        lead = (case["B"],) if op == "ssm_step" else (case["T"],) if op == "ssm_prompt" else (case["B"], case["T"])
        xz = randn(*lead, 2 * -(-D // 8) * 8)          # one projection gives x and z
        s["x"], s["z"] = xz[..., :D], xz[..., xz.shape[-1] // 2:][..., :D]
        s["dt"] = randn(*lead, D, scale=0.5)
        bc = randn(*lead, 2 * G * N)                    # and one B and C
        s["B"] = bc[..., :G * N].unflatten(-1, (G, N))
        s["C"] = bc[..., G * N:].unflatten(-1, (G, N))
        # time steps of 0.001 to 0.1 before the inputs move them, decays of 1 .. N: the usual initialisation
        step = torch.exp(rand(D) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * (0.9 + 0.2 * rand(D, 1))
        s["Dk"] = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
        if op == "ssm_step":
            S, s["slots"] = pool(case["B"])
            s["h"] = randn(S, D, N, scale=0.1, dtype=torch.float32)
        elif op == "ssm_prompt":
            s["h"] = randn(case["seqs"], D, N, scale=0.1, dtype=torch.float32)
        else:
            s["dy"] = randn(*lead, D)
    else:
        B, H, HV = case["B"], case["H"], case["HV"]
        S, s["slots"] = pool(B)
        q, k = (torch.randn(B, H, 128, generator=gen, device="cuda") for _ in range(2))
        s["q"], s["k"] = ((t / t.norm(dim=-1, keepdim=True)).to(io) for t in (q, k))
        s["v"], s["beta"] = randn(B, HV, 128), rand(B, HV).to(io)
        g = torch.randn(*((B, HV, 128) if case["per_k"] else (B, HV)), generator=gen, device="cuda")
        s["g"] = torch.nn.functional.logsigmoid(g) / 16
        s["h"] = randn(S, HV, 128, 128, scale=0.1, dtype=torch.float32)
    if op in ("conv_prompt", "ssm_prompt"):
        s["cu"] = torch.tensor([0] + lengths(case)).cumsum(0).to(torch.int32).cuda()
    return s


# ---------------------------------------------------------------- plain forms (32 bits, rounded once at the end)

def _silu(x):
    return x * torch.sigmoid(x)


def _plain_norm8(s):
    s32 = s["x"].float() + s["res"].float()
    y = s32 * torch.rsqrt((s32 * s32).mean(-1, keepdim=True) + EPS) * s["w"].float()
    rows, D = y.shape
    group = s["case"]["group"] or D
    pad = torch.nn.functional.pad(y, (0, -D % group)).unflatten(-1, (-1, group))
    scale = (pad.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    y8 = (pad / scale[..., None]).flatten(1)[:, :D].to(torch.float8_e4m3fn)
    return dict(r=s32.to(s["x"].dtype), y8=y8, scale=scale)


def _plain_norm_train(s):
    io, w, dy = s["x"].dtype, s["w"].float(), s["dy"].float()
    s32 = s["x"].float() + s["res"].float()
    y = s32 * torch.rsqrt((s32 * s32).mean(-1, keepdim=True) + EPS) * w
    r = s32.to(io)
    r32 = r.float()                                     # the backward reads r as it was kept
    rstd = torch.rsqrt((r32 * r32).mean(-1, keepdim=True) + EPS)
    xh, wdy = r32 * rstd, dy * w
    dx = rstd * (wdy - xh * (wdy * xh).mean(-1, keepdim=True)) + s["dr"].float()
    return dict(y=y.to(io), r=r, dx=dx.to(io), dw=(dy * xh).sum(0))


def _plain_conv(x, state, cu, w, b):
    """x [T, D] packed, state [n, W - 1, D] fp32 -> the preactivations, the windows [T, W, D] and the new states."""
    T, D = x.shape
    n, back = cu.numel() - 1, w.shape[1] - 1
    cu = cu.long()
    rows = torch.cat([x, state.reshape(n * back, D)])

    def row_of(seq, token):      # a token of the sequence, or of its state where it lies before the start
        before = token - cu[seq]
        return torch.where(before >= 0, token, T + seq * back + back + before)

    t = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    taps = torch.arange(back + 1, device=x.device) - back
    win = rows[row_of(seq[:, None].expand(-1, back + 1), t[:, None] + taps)]
    pre = (win * w.t()).sum(1) + b
    last = cu[1:, None] + torch.arange(back, device=x.device) - back
    return pre, win, rows[row_of(torch.arange(n, device=x.device)[:, None].expand(-1, back), last)]


def _plain_conv_prompt(s):
    io = s["x"].dtype
    pre, _, state = _plain_conv(s["x"].float(), s["state"].float(), s["cu"], s["w"].float(), s["b"].float())
    return dict(y=_silu(pre).to(io), state=state.to(io))


def _plain_conv_train(s):
    io, (B, T, D), w = s["x"].dtype, s["x"].shape, s["w"].float()
    cu = torch.arange(B + 1, device="cuda") * T
    pre, win, _ = _plain_conv(s["x"].float().flatten(0, 1), torch.zeros(B, TAPS - 1, D, device="cuda"), cu, w,
                              s["b"].float())
    sig = torch.sigmoid(pre)
    dp = s["dy"].float().flatten(0, 1) * sig * (1 + pre * (1 - sig))
    ahead = torch.nn.functional.pad(dp.view(B, T, D), (0, 0, 0, TAPS - 1)).unfold(1, TAPS, 1)     # [B, T, D, W]
    dx = (ahead * w.flip(1)).sum(-1)
    return dict(y=(pre * sig).to(io).view(B, T, D), dx=dx.to(io), dw=(dp[:, None] * win).sum(0).t().contiguous(),
                db=dp.sum(0))


def _pick(pool, slots):
    """The rows of a pool at the slots; padding reads the last slot, which is nobody's."""
    at = torch.where(slots < 0, pool.shape[0] - 1, slots).long()
    return at, pool[at]


def _plain_conv_step(s):
    ok = (s["slots"] >= 0)[:, None]
    at, old = _pick(s["state"], s["slots"])
    win = torch.cat([old, s["x"][:, None]], 1)
    y = _silu((win.float() * s["w"].float().t()).sum(1) + s["b"].float())
    s["state"][at] = torch.where(ok[..., None], win[:, 1:], old)
    return dict(y=torch.where(ok, y, 0).to(s["x"].dtype), state=s["state"])


def _plain_delta(s):
    return torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])


def _spread(bc, D):
    """B or C of a group for each of its channels."""
    return bc.float().repeat_interleave(D // bc.shape[-2], -2)


def _scan(a, b, dim):
    """h_t = a_t h_{t-1} + b_t along `dim`, from zero: doubles the reach in each step (in place)."""
    T, reach = a.shape[dim], 1
    while reach < T:
        late, early = (lambda v: v.narrow(dim, reach, T - reach)), (lambda v: v.narrow(dim, 0, T - reach))
        late(b).add_(late(a) * early(b))
        late(a).copy_(late(a) * early(a))
        reach *= 2
    return b


def _plain_ssm_prompt(s):
    io, x, cu, (T, D) = s["x"].dtype, s["x"].float(), s["cu"].long(), s["x"].shape
    dl = _plain_delta(s)
    seq = torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True) - 1
    first = (torch.arange(T, device="cuda") == cu[seq])[:, None, None]
    a = torch.exp(dl[..., None] * s["A"])
    b = (dl * x)[..., None] * _spread(s["B"], D)
    b += torch.where(first, a * s["h"][seq], 0)
    h = _scan(a.masked_fill_(first, 0.0), b, 0)
    y = ((h * _spread(s["C"], D)).sum(-1) + s["Dk"] * x) * _silu(s["z"].float())
    some = (cu[1:] > cu[:-1])[:, None, None]
    return dict(y=y.to(io), h=torch.where(some, h[(cu[1:] - 1).clamp_min(0)], s["h"]))


def _plain_ssm_train(s):
    io, x, z, dy, D = s["x"].dtype, s["x"].float(), s["z"].float(), s["dy"].float(), s["x"].shape[-1]
    raw = s["dt"].float() + s["dt_bias"]
    dl = torch.nn.functional.softplus(raw)
    Bs, Cs = _spread(s["B"], D), _spread(s["C"], D)
    a = torch.exp(dl[..., None] * s["A"])
    h = _scan(a.clone(), (dl * x)[..., None] * Bs, 1)
    ah = torch.cat([torch.zeros_like(h[:, :1]), a[:, 1:] * h[:, :-1]], 1)          # a_t h_{t-1}
    pre = (h * Cs).sum(-1) + s["Dk"] * x
    sig = torch.sigmoid(z)
    dpre = dy * z * sig
    dz = dy * pre * sig * (1 + z * (1 - sig))
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)                   # a_{t+1}
    dh = _scan(after.flip(1), (dpre[..., None] * Cs).flip(1), 1).flip(1)
    dlx = (dh * Bs).sum(-1)
    dlog = dh * ah
    ddl = dlx * x + (dlog * s["A"]).sum(-1)
    draw_ = ddl * torch.sigmoid(raw)
    groups = (s["B"].shape[-2], -1)
    dB = (dh * (dl * x)[..., None]).unflatten(2, groups).sum(3)
    dC = (h * dpre[..., None]).unflatten(2, groups).sum(3)
    return dict(y=(pre * z * sig).to(io), h=h[:, -1], dx=(dlx * dl + s["Dk"] * dpre).to(io), ddt=draw_.to(io),
                dA=(dlog * dl[..., None]).sum((0, 1)), dB=dB.to(io), dC=dC.to(io), dD=(dpre * x).sum((0, 1)),
                dz=dz.to(io), dbias=draw_.sum((0, 1)))


def _plain_ssm_step(s):
    D, x = s["x"].shape[-1], s["x"].float()
    ok = (s["slots"] >= 0)[:, None]
    at, old = _pick(s["h"], s["slots"])
    dl = _plain_delta(s)
    h = torch.exp(dl[..., None] * s["A"]) * old + (dl * x)[..., None] * _spread(s["B"], D)
    y = ((h * _spread(s["C"], D)).sum(-1) + s["Dk"] * x) * _silu(s["z"].float())
    s["h"][at] = torch.where(ok[..., None], h, old)
    return dict(y=torch.where(ok, y, 0).to(s["x"].dtype), h=s["h"])


def _plain_delta_step(s):
    case, io = s["case"], s["q"].dtype
    ok = (s["slots"] >= 0)[:, None, None]
    at, old = _pick(s["h"], s["slots"])
    q, k = (s[n].float().repeat_interleave(case["HV"] // case["H"], 1)[..., None] for n in ("q", "k"))
    decay = torch.exp(s["g"])
    h = old * (decay[..., None] if case["per_k"] else decay[..., None, None])
    delta = s["beta"].float()[..., None] * (s["v"].float() - (h * k).sum(-2))
    h = h + k * delta[..., None, :]
    o = (h * q).sum(-2) / math.sqrt(128)
    s["h"][at] = torch.where(ok[..., None], h, old)
    return dict(o=torch.where(ok, o, 0).to(io), h=s["h"])


# ---------------------------------------------------------------- the library's calls

def _own(s):
    from chunked_gated_delta_prepare_gb300 import layer
    op = s["op"]
    if op == "norm8":
        _, r, y8, scale = layer.norm_forward(s["x"], s["w"], s["res"], eps=EPS, quant=s["case"]["group"] or "row",
                                             want_y=False)
        return dict(r=r, y8=y8, scale=scale)
    if op == "norm_train":
        y, r, _, _ = layer.norm_forward(s["x"], s["w"], s["res"], eps=EPS)
        dx, dw = layer.norm_backward(s["dy"], r, s["w"], s["dr"], eps=EPS)
        return dict(y=y, r=r, dx=dx, dw=dw)
    if op == "conv_prompt":
        y, state = layer.conv_forward(s["x"], s["w"], s["b"], s["state"], cu_seqlens=s["cu"])
        return dict(y=y, state=state)
    if op == "conv_train":
        y, _ = layer.conv_forward(s["x"], s["w"], s["b"], want_state=False)
        dx, dw, db, _ = layer.conv_backward(s["x"], s["w"], s["b"], s["dy"])
        return dict(y=y, dx=dx, dw=dw, db=db)
    if op == "conv_step":
        return dict(y=layer.conv_step(s["x"], s["w"], s["b"], s["state"], slots=s["slots"]), state=s["state"])
    if op == "delta_step":
        o = layer.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"], slots=s["slots"])
        return dict(o=o, h=s["h"])
    five = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = dict(D=s["Dk"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "ssm_step":
        return dict(y=layer.ssm_step(*five, s["h"], slots=s["slots"], **more), h=s["h"])
    if op == "ssm_prompt":
        y, h = layer.ssm_forward(*five, h0=s["h"], cu_seqlens=s["cu"], **more)
        return dict(y=y, h=h)
    y, h = layer.ssm_forward(*five, **more)
    d = layer.ssm_backward(*five, s["dy"], **more)
    return dict(y=y, h=h, dx=d.dx, ddt=d.ddt, dA=d.dA, dB=d.dB, dC=d.dC, dD=d.dD, dz=d.dz, dbias=d.ddt_bias)


PLAIN = dict(norm8=_plain_norm8, norm_train=_plain_norm_train, conv_prompt=_plain_conv_prompt,
             conv_train=_plain_conv_train, conv_step=_plain_conv_step, ssm_prompt=_plain_ssm_prompt,
             ssm_train=_plain_ssm_train, ssm_step=_plain_ssm_step, delta_step=_plain_delta_step)


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass has to move and compute

def work(case):
    op, e = case["op"], ES[case["io"]]
    D = case.get("D", 0)
    if op == "norm8":
        n, scales = case["rows"] * D, case["rows"] * (-(-D // (case["group"] or D)))
        return dict(bytes=n * (3 * e + 1) + 4 * scales + D * e, flops=7 * n)
    if op == "norm_train":                              # x, res, y, r; r, dy, dr, dx
        n = case["rows"] * D
        return dict(bytes=8 * n * e + D * (2 * e + 4), flops=16 * n)
    if op == "conv_prompt":
        n = case["T"] * D
        return dict(bytes=2 * n * e + case["seqs"] * 2 * (TAPS - 1) * D * e + 5 * D * e, flops=(2 * TAPS + 5) * n)
    if op == "conv_train":                              # x, y; x, dy, dx
        n = case["B"] * case["T"] * D
        return dict(bytes=5 * n * e + D * (TAPS + 1) * (2 * e + 4), flops=(8 * TAPS + 16) * n)
    if op == "conv_step":
        n = case["B"] * D
        return dict(bytes=2 * TAPS * n * e + 5 * D * e, flops=(2 * TAPS + 5) * n)
    if op == "delta_step":
        B, H, HV = case["B"], case["H"], case["HV"]
        vectors = B * e * (2 * H * 128 + 2 * HV * 128 + HV) + 4 * B * HV * (128 if case["per_k"] else 1)
        return dict(bytes=2 * 4 * B * HV * 128 * 128 + vectors, flops=7 * B * HV * 128 * 128)
    N, G = case["N"], case["G"]
    n = case["B"] * D if op == "ssm_step" else case["T"] * D * (case["B"] if op == "ssm_train" else 1)
    bc, fixed = 2 * (n // D) * G * N * e, 4 * D * (N + 2)
    if op == "ssm_train":                               # x, dt, z, y; x, dt, z, dy, dx, ddt, dz; B, C twice, dB, dC
        return dict(bytes=11 * n * e + 3 * bc + 3 * fixed + 4 * case["B"] * D * N, flops=29 * n * N + 40 * n)
    states = 2 * 4 * (case["B"] if op == "ssm_step" else case["seqs"]) * D * N
    return dict(bytes=4 * n * e + bc + fixed + states, flops=7 * n * N + 12 * n)


# ---------------------------------------------------------------- the definition in 64 bits

def _d(t):
    return t.double()


def _sig64(x):
    return 1 / (1 + torch.exp(-x))


def _exact_norm(s, case):
    x = _d(s["x"]) + _d(s["res"])
    r = x.to(s["x"].dtype)
    w = _d(s["w"])
    y = x / torch.sqrt(x.pow(2).mean(1) + EPS)[:, None] * w
    if case["op"] == "norm8":
        rows, D = y.shape
        width = case["group"] or D
        scale = torch.stack([y[:, at:at + width].abs().max(1).values / 448 for at in range(0, D, width)], 1)
        per = scale.repeat_interleave(width, 1)[:, :D]
        return dict(r=_d(r), y8=y / per, scale=scale)
    r = _d(r)
    norm = torch.sqrt(r.pow(2).mean(1) + EPS)[:, None]
    dy, dr = _d(s["dy"]), _d(s["dr"])
    dot = (dy * w * r).mean(1)[:, None]
    return dict(y=y, r=r, dx=dy * w / norm - r * dot / norm ** 3 + dr, dw=(dy * r / norm).sum(0))


def _conv64(xs, state, w, b):
    """One sequence: xs [L, D] after state [W - 1, D]; the preactivations and all the rows."""
    rows = torch.cat([state, xs])
    pre = b.expand(xs.shape).clone()
    for j in range(w.shape[1]):
        pre += w[:, j] * rows[j:j + xs.shape[0]]
    return pre, rows


def _exact_conv(s, case):
    w, b = _d(s["w"]), _d(s["b"])
    back = TAPS - 1
    if case["op"] == "conv_prompt":
        ys, states, at = [], [], 0
        for i, n in enumerate(lengths(case)):
            pre, rows = _conv64(_d(s["x"][at:at + n]), _d(s["state"][i]), w, b)
            ys.append(pre * _sig64(pre))
            states.append(rows[n:])
            at += n
        return dict(y=torch.cat(ys), state=torch.stack(states))
    if case["op"] == "conv_step":
        y, state = torch.zeros_like(_d(s["x"])), _d(s["state"])
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                pre, rows = _conv64(_d(s["x"][i:i + 1]), state[slot], w, b)
                y[i], state[slot] = (pre * _sig64(pre))[0], rows[1:]
        return dict(y=y, state=state)
    ys, dxs, dw, db = [], [], torch.zeros_like(w), torch.zeros_like(b)
    for x, dy in zip(_d(s["x"]), _d(s["dy"])):
        T = x.shape[0]
        pre, rows = _conv64(x, torch.zeros_like(x[:1]).expand(back, -1), w, b)
        sg = _sig64(pre)
        dp = dy * (sg + pre * sg * (1 - sg))
        drows = torch.zeros_like(rows)
        for j in range(TAPS):
            drows[j:j + T] += w[:, j] * dp
            dw[:, j] += (dp * rows[j:j + T]).sum(0)
        db += dp.sum(0)
        ys.append(pre * sg)
        dxs.append(drows[back:])
    return dict(y=torch.stack(ys), dx=torch.stack(dxs), dw=dw, db=db)


def _exact_ssm(s, case):
    op, G, D = case["op"], case["G"], case["D"]
    per = D // G
    x, z, A, Dk = _d(s["x"]), _d(s["z"]), _d(s["A"]), _d(s["Dk"])
    raw = _d(s["dt"]) + _d(s["dt_bias"])
    dl = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    Bm, Cm = _d(s["B"]), _d(s["C"])

    def wide(v):                     # [..., G, N] -> [..., D, N]
        return v[..., :, None, :].expand(*v.shape[:-1], per, v.shape[-1]).reshape(*v.shape[:-2], D, v.shape[-1])

    gate = z * _sig64(z)
    if op == "ssm_step":
        y, h = torch.zeros_like(x), _d(s["h"])
        at = s["slots"].long()
        new = torch.exp(dl[..., None] * A) * h[at] + (dl * x)[..., None] * wide(Bm)
        y = ((new * wide(Cm)).sum(-1) + Dk * x) * gate * (at >= 0)[:, None]
        h[at[at >= 0]] = new[at >= 0]
        return dict(y=y, h=h)
    if op == "ssm_prompt":
        pre, last, at = torch.empty_like(x), [], 0
        for i, n in enumerate(lengths(case)):
            h = _d(s["h"][i])
            for t in range(at, at + n):
                h = torch.exp(dl[t][:, None] * A).mul_(h).add_((dl[t] * x[t])[:, None] * wide(Bm[t]))
                pre[t] = (h * wide(Cm[t])).sum(-1)
            last.append(h)
            at += n
        return dict(y=(pre + Dk * x) * gate, h=torch.stack(last))
    nb, T = x.shape[:2]
    h = x.new_zeros(nb, D, case["N"])
    hs = [h]
    for t in range(T):
        h = torch.exp(dl[:, t, :, None] * A) * h + (dl[:, t] * x[:, t])[..., None] * wide(Bm[:, t])
        hs.append(h)
    pre = torch.stack([(hs[t + 1] * wide(Cm[:, t])).sum(-1) for t in range(T)], 1) + Dk * x
    dy, sz = _d(s["dy"]), _sig64(z)
    dpre = dy * gate
    dx, ddl, dA, dB, dC = Dk * dpre, torch.zeros_like(x), torch.zeros_like(A), torch.zeros_like(Bm), torch.zeros_like(Cm)
    dh = torch.zeros_like(h)
    for t in range(T - 1, -1, -1):
        dh = dh + dpre[:, t, :, None] * wide(Cm[:, t])
        dC[:, t] = (hs[t + 1] * dpre[:, t, :, None]).reshape(nb, G, per, -1).sum(2)
        dB[:, t] = (dh * (dl[:, t] * x[:, t])[..., None]).reshape(nb, G, per, -1).sum(2)
        through = (dh * wide(Bm[:, t])).sum(-1)
        decay = torch.exp(dl[:, t, :, None] * A)
        dlog = dh * decay * hs[t]
        dx[:, t] += through * dl[:, t]
        ddl[:, t] = through * x[:, t] + (dlog * A).sum(-1)
        dA += (dlog * dl[:, t, :, None]).sum(0)
        dh = dh * decay
    ddt = ddl * _sig64(raw)
    return dict(y=pre * gate, h=hs[-1], dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(dpre * x).sum((0, 1)),
                dz=dy * pre * (sz + z * sz * (1 - sz)), dbias=ddt.sum((0, 1)))


def _exact_delta(s, case):
    o, h = torch.zeros_like(_d(s["v"])), _d(s["h"])
    per = case["HV"] // case["H"]
    for i, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        q, k = (_d(s[n][i]).repeat_interleave(per, 0) for n in ("q", "k"))
        decay = torch.exp(_d(s["g"][i]))
        S = h[slot] * (decay[..., None] if case["per_k"] else decay[:, None, None])
        delta = _d(s["beta"][i])[:, None] * (_d(s["v"][i]) - torch.einsum("hkv,hk->hv", S, k))
        S = S + k[:, :, None] * delta[:, None, :]
        h[slot], o[i] = S, torch.einsum("hkv,hk->hv", S, q) / math.sqrt(128)
    return dict(o=o, h=h)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(s, case)
    if op.startswith("conv"):
        return _exact_conv(s, case)
    if op.startswith("ssm"):
        return _exact_ssm(s, case)
    return _exact_delta(s, case)
