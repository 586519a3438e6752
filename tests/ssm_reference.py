"""The selective state space scan in 64 bits, token by token, with the sizes of its terms (plain torch, any device)."""
import torch


def spread(bc, D):
    """B or C [..., G, N] for each channel [..., D, N]."""
    return bc.double().repeat_interleave(D // bc.shape[-2], -2)


def scan(x, dt, A, B, C, Dk=None, z=None, bias=None, h0=None, softplus=True):
    """One sequence [T, D]: y, the last state, all states [T + 1, D, N], and the sizes of y's and the states' terms."""
    T, D = x.shape
    x, A = x.double(), A.double()
    raw = dt.double() + (bias.double() if bias is not None else 0)
    dl = torch.nn.functional.softplus(raw, threshold=200) if softplus else raw
    B, C = spread(B, D), spread(C, D)
    h = h0.double().clone() if h0 is not None else torch.zeros(A.shape, device=x.device, dtype=torch.double)
    size = h.abs()
    hs, sizes = [h], [size]
    for t in range(T):
        a = torch.exp(dl[t][:, None] * A)
        h = a * h + (dl[t] * x[t])[:, None] * B[t]
        size = a * size + (dl[t] * x[t]).abs()[:, None] * B[t].abs()
        hs.append(h)
        sizes.append(size)
    hs, sizes = torch.stack(hs), torch.stack(sizes)
    y, ysize = (hs[1:] * C).sum(-1), (sizes[1:] * C.abs()).sum(-1)
    if Dk is not None:
        y, ysize = y + Dk.double() * x, ysize + (Dk.double() * x).abs()
    if z is not None:
        gate = z.double() * torch.sigmoid(z.double())
        y, ysize = y * gate, ysize * gate.abs()
    return y, hs[-1], hs, ysize, sizes


def scan_backward(x, dt, A, B, C, dy, Dk=None, z=None, bias=None, h0=None, dh_final=None, softplus=True):
    """One sequence: {name: (gradient, size of its terms)} of y and the last state, by the reverse recurrence."""
    T, D = x.shape
    _, _, hs, _, hsize = scan(x, dt, A, B, C, None, None, bias, h0, softplus)
    G, N = B.shape[-2:]
    x64, A64, dy64 = x.double(), A.double(), dy.double()
    raw = dt.double() + (bias.double() if bias is not None else 0)
    dl = torch.nn.functional.softplus(raw, threshold=200) if softplus else raw
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    Bs, Cs = spread(B, D), spread(C, D)
    if z is not None:
        sig = torch.sigmoid(z.double())
        gate, dgate = z.double() * sig, sig * (1 + z.double() * (1 - sig))
    else:
        gate = torch.ones_like(x64)
    g = dy64 * gate
    dh = dh_final.double().clone() if dh_final is not None else torch.zeros_like(hs[0])
    ds = dh.abs()
    zero = lambda *s: [torch.zeros(*s, device=x.device, dtype=torch.double) for _ in range(2)]  # noqa: E731
    out = {"dx": zero(T, D), "ddt": zero(T, D), "dB": zero(T, G, N), "dC": zero(T, G, N), "dA": zero(D, N)}
    for t in range(T - 1, -1, -1):
        a = torch.exp(dl[t][:, None] * A64)
        dh, ds = dh + g[t][:, None] * Cs[t], ds + g[t].abs()[:, None] * Cs[t].abs()
        u = dl[t] * x64[t]
        out["dC"][0][t] = (g[t][:, None] * hs[t + 1]).view(G, -1, N).sum(1)
        out["dC"][1][t] = (g[t].abs()[:, None] * hsize[t + 1]).view(G, -1, N).sum(1)
        out["dB"][0][t] = (dh * u[:, None]).view(G, -1, N).sum(1)
        out["dB"][1][t] = (ds * u.abs()[:, None]).view(G, -1, N).sum(1)
        r, rs = (dh * Bs[t]).sum(-1), (ds * Bs[t].abs()).sum(-1)
        w, ws = dh * a * hs[t], ds * a * hsize[t]
        out["dx"][0][t], out["dx"][1][t] = r * dl[t], rs * dl[t]
        out["ddt"][0][t] = (r * x64[t] + (A64 * w).sum(-1)) * slope[t]
        out["ddt"][1][t] = (rs * x64[t].abs() + (A64.abs() * ws).sum(-1)) * slope[t]
        out["dA"][0] += dl[t][:, None] * w
        out["dA"][1] += dl[t][:, None] * ws
        dh, ds = a * dh, a * ds
    out["dh0"] = [dh, ds]
    out["ddt_bias"] = [v.sum(0) for v in out["ddt"]]
    pre, pres = (hs[1:] * Cs).sum(-1), (hsize[1:] * Cs.abs()).sum(-1)
    if Dk is not None:
        out["dx"][0] += Dk.double() * g
        out["dx"][1] += (Dk.double() * g).abs()
        out["dD"] = [(g * x64).sum(0), (g * x64).abs().sum(0)]
        pre, pres = pre + Dk.double() * x64, pres + (Dk.double() * x64).abs()
    if z is not None:      # silu' = sig + z sig (1 - sig): where its terms cancel its error is theirs
        out["dz"] = [dy64 * pre * dgate, dy64.abs() * pres * (sig + (z.double() * sig * (1 - sig)).abs())]
    return out
