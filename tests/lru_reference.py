"""The gated linear recurrence in 64 bits, token by token, with the sizes of its terms (plain torch, any device)."""
import torch


def gates(x, r, i=None, lam=None, c=8.0):
    """The decay, the input's part, the input's gate, sigmoid(r), 1 - sigmoid(r), and a channel's rate (or None)."""
    x, r = x.double(), r.double()
    q, rest = torch.sigmoid(r), torch.sigmoid(-r)
    g = torch.sigmoid(i.double()) if i is not None else torch.ones_like(x)
    if lam is None:
        return q, rest, g, q, rest, None
    lam = lam.double()
    k = c * (lam.clamp_min(0) + torch.log1p(torch.exp(-lam.abs())))
    return torch.exp(-k * q), torch.sqrt(-torch.expm1(-2 * k * q)), g, q, rest, k


def scan(x, r, i=None, lam=None, h0=None, c=8.0):
    """One sequence [T, D]: all states [T + 1, D] and the sizes of their terms."""
    a, s, g, *_ = gates(x, r, i, lam, c)
    u = s * g * x.double()
    h = h0.double().clone() if h0 is not None else torch.zeros(x.shape[1], device=x.device, dtype=torch.double)
    hs, sizes = [h], [h.abs()]
    for t in range(x.shape[0]):
        hs.append(a[t] * hs[-1] + u[t])
        sizes.append(a[t] * sizes[-1] + u[t].abs())
    return torch.stack(hs), torch.stack(sizes)


def scan_backward(x, r, i, lam, dy, h0=None, dh_final=None, c=8.0):
    """One sequence: {name: (gradient, size of its terms)} of y and the last state, by the reverse recurrence."""
    a, s, g, q, rest, k = gates(x, r, i, lam, c)
    hs, hsize = scan(x, r, i, lam, h0, c)
    x, dy = x.double(), dy.double()
    e, es = torch.zeros_like(x), torch.zeros_like(x)
    run = dh_final.double().clone() if dh_final is not None else torch.zeros(x.shape[1], device=x.device).double()
    size = run.abs()
    for t in range(x.shape[0] - 1, -1, -1):
        e[t], es[t] = run + dy[t], size + dy[t].abs()
        run, size = e[t] * a[t], es[t] * a[t]
    before, bsize = hs[:-1], hsize[:-1]
    out = {"dx": (e * s * g, es * s * g), "dh0": (run, size)}
    if i is not None:
        out["di"] = tuple(v * s * g * torch.sigmoid(-i.double()) for v in (e * x, es * x.abs()))
    if lam is None:
        out["dr"] = (e * (before - g * x) * a * s, es * (bsize + g * x.abs()) * a * s)
        return out
    # q / s stays finite where both are zero: their limit there is zero
    ratio = torch.where(s > 0, a / s.clamp_min(1e-300), torch.zeros_like(s))
    dlog, dsize = e * a * (before - g * x * ratio), es * a * (bsize + g * x.abs() * ratio)
    slope = c * torch.sigmoid(lam.double())
    out["dr"] = (-dlog * k * q * rest, dsize * k * q * rest)
    out["dlam"] = (-(dlog * q).sum(0) * slope, (dsize * q).sum(0) * slope)
    return out
