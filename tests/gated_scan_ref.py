"""The gated linear recurrence and its gradients in 64 bits, token by token, and how far the
kernels' 32-bit sums may be from them.

The bounds follow an error through the recurrence.  With e = 2^-24 (half a unit of fp32, a
hardware exp2, reciprocal or square root is off by at most two of it):
 - sigmoid(z): e^-z takes its argument rounded (|z| e relative, halved by the precise form but
   counted whole) and an exp2, an add, a reciprocal: (|z| + 6) e;
 - a = e^-v: v's own error times v, and 3 e;
 - b = 1 - a: a's 2 e over b >= 0.11 where it is a difference (16 e), below its series; the root
   of b (2 - b) has half of that and 3 e: m is off by (12 + (|r| + 6)) e;
 - what a token adds, m sigmoid(i) x: (24 + |r| + |i|) e |u|;
 - a step: the state's own error times a, 5 e of the sum of magnitudes for the factor and the
   rounding, and v's error (|r| + 6) e v of the state before;
 - the joins over waves and chunks: at most 16 in a block, 8 + 4 before it and one group, each a
   step of the kind above: 64 e of the sum of magnitudes, and as much again once in 128 tokens
   (half an e per token).
"""
import torch

E = 2.0 ** -24


def gates(x, r, i, decay):
    x, r, i, decay = (t.double() for t in (x, r, i, decay))
    sr, g = torch.sigmoid(r), torch.sigmoid(i)
    v = decay * sr
    m = torch.sqrt(-torch.expm1(-2.0 * v))
    return v, sr, g, m, x


def masks(shape, seq_lens, reset, device):
    B, L, _ = shape
    live = torch.ones((B, L), dtype=torch.bool, device=device)
    if seq_lens is not None:
        live = torch.arange(L, device=device) < seq_lens.to(device).long()[:, None]
    on = live.clone() if reset is None else live & (reset.to(device) == 0)
    return live, on


def forward(x, r, i, decay, h0=None, seq_lens=None, reset=None):
    """A dict: y, last_state, states, and y_bound, last_bound (fp32 errors, no output rounding)."""
    B, L, dim = x.shape
    live, on = masks(x.shape, seq_lens, reset, x.device)
    x = torch.where(live[..., None], x, torch.zeros_like(x))  # padding may hold anything
    r = torch.where(live[..., None], r, torch.zeros_like(r))
    i = torch.where(live[..., None], i, torch.zeros_like(i))
    v, sr, g, m, xd = gates(x, r, i, decay)
    a, u = torch.exp(-v), m * g * xd
    er, ei = r.double().abs() + 6.0, i.double().abs() + 6.0
    h = torch.zeros((B, dim), dtype=torch.float64, device=x.device) if h0 is None else h0.double().clone()
    big, err = h.abs(), torch.zeros_like(h)
    y, yb, before, bb = [], [], [], []
    for t in range(L):
        before.append(h)
        bb.append(err + 64 * E * big)
        lt, ot = live[:, t, None], on[:, t, None]
        hp, bp, ep = (torch.where(ot, z, torch.zeros_like(z)) for z in (h, big, err))
        nb = a[:, t] * bp + u[:, t].abs()
        ne = a[:, t] * ep + E * (5.5 * nb + er[:, t] * v[:, t] * bp + (12 + er[:, t] + ei[:, t]) * u[:, t].abs())
        h = torch.where(lt, a[:, t] * hp + u[:, t], h)
        big, err = torch.where(lt, nb, big), torch.where(lt, ne, err)
        y.append(torch.where(lt, h, torch.zeros_like(h)))
        yb.append(torch.where(lt, err + 64 * E * big + 1e-36, torch.zeros_like(h)))

    def stack(z):
        return torch.stack(z, 1) if z else torch.zeros((B, 0, dim), dtype=torch.float64, device=x.device)
    return dict(y=stack(y), y_bound=stack(yb), last_state=h, last_bound=err + 64 * E * big + 1e-36,
                before=stack(before), before_bound=stack(bb), live=live, on=on, x=x, r=r, i=i)


def backward(x, r, i, decay, dy, dlast=None, h0=None, seq_lens=None, reset=None):
    """A dict of gradients, and NAME_bound for each."""
    f = forward(x, r, i, decay, h0, seq_lens, reset)
    live, on = f["live"], f["on"]
    v, sr, g, m, xd = gates(f["x"], f["r"], f["i"], decay)
    er, ei = f["r"].double().abs() + 6.0, f["i"].double().abs() + 6.0
    a = torch.exp(-v)
    B, L, dim = x.shape
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    dy = torch.where(live[..., None], dy.double(), zero)
    c = torch.zeros((B, dim), dtype=torch.float64, device=x.device) if dlast is None else dlast.double().clone()
    big, err = c.abs(), torch.zeros_like(c)
    lam, lb = torch.zeros_like(dy), torch.zeros_like(dy)
    lbig = torch.zeros_like(dy)
    for t in range(L - 1, -1, -1):
        lt, ot = live[:, t, None], on[:, t, None]
        lam[:, t] = torch.where(lt, dy[:, t] + c, zero)
        nb = dy[:, t].abs() + big
        lbig[:, t] = torch.where(lt, nb, zero)
        lb[:, t] = torch.where(lt, err + E * 65 * nb, zero)
        ne = a[:, t] * (err + 5.5 * E * nb) + E * er[:, t] * v[:, t] * nb
        c = torch.where(lt, torch.where(ot, a[:, t] * lam[:, t], zero), c)
        big = torch.where(lt, torch.where(ot, a[:, t] * nb, zero), big)
        err = torch.where(lt, torch.where(ot, ne, zero), err)
    h = torch.where(on[..., None], f["before"], zero)
    hb = torch.where(on[..., None], f["before_bound"], zero)
    safe = torch.where(m > 0, m, torch.ones_like(m))
    avm = a * torch.where(m > 0, v / safe, torch.zeros_like(v))
    one, two = g * xd * avm, v * h
    P = lam * a * (one - two)
    dx, di = lam * m * g, lam * m * xd * g * (1 - g)
    dr = P * (1 - sr)
    k = 30 + er + ei
    # a's relative error is v's absolute one, er E v, and a stands in `one` a second time: with
    # v of 20 and more (decay 300) that is past the other terms
    kp = k + er * v
    Pb = (lb * a * (one - two).abs() + lbig * a * (v * hb + 2 * kp * E * (one.abs() + two.abs())))
    # an a below 2^-126 is 0 in 32 bits, times v (88 there) and the state: past the 1e-36 below
    Pb = Pb + 2.0 ** -126 * lbig * v * h.abs()
    out = dict(dx=dx, dr=dr, di=di, dh0=c, ddecay=P.sum((0, 1)) / decay.double())
    out.update(dx_bound=(lb + lbig * k * E) * m * g + 1e-36,
               di_bound=(lb + lbig * k * E) * m * (xd * g * (1 - g)).abs() + 1e-36,
               dr_bound=(Pb + 2 * er * E * P.abs()) * (1 - sr) + 1e-36,
               dh0_bound=err + 64 * E * big + 1e-36,
               # 128 terms of a chunk in fp32, 8 of a thread and 16 of its waves
               ddecay_bound=(Pb + 24 * E * P.abs()).sum((0, 1)) / decay.double() + E * (P.sum((0, 1)) / decay.double()).abs() + 1e-36)
    return out


def rounding(io):
    """Half a unit of the output's type, relative."""
    return torch.finfo(io).eps / 2


def check(name, got, want, bound, io=torch.float32):
    err = (got.double() - want).abs()
    most = bound + rounding(io) * (want.abs() + bound)
    ratio = torch.where(err == 0, torch.zeros_like(err), err / most)  # 0 / 0 where both are exact
    worst = ratio.max().item() if err.numel() else 0.0
    assert torch.isfinite(got).all(), f"{name}: not finite"
    assert worst <= 1.0, f"{name}: {worst:.2f} times the bound, largest error {err.max().item():.3e}"
    return worst
