"""Residual + dropout + norm, dropout and rotary positions in 64 bits, and how far the kernels'
32-bit arithmetic may be from them (e = 2^-24: one rounding).

Sums of a row: a lane adds up to 16 values, then six shuffles and up to 16 waves: 40 e of the
sum of magnitudes.  The generator is written in Python's whole numbers.
"""
import numpy as np
import torch

E = 2.0 ** -24


def philox(counter, key):
    """Philox4x32 with ten rounds: four counter words (arrays of uint64 below 2^32), two key words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(w, dtype=np.uint64) for w in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & low,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def words(rng, site, start, n):
    """Words start .. start + n - 1 of the stream (rng, site)."""
    seed, offset = (int(t) & (1 << 64) - 1 for t in rng.tolist())
    offset = (offset + site) & (1 << 64) - 1
    first = start // 4
    j = np.arange(first, (start + n + 3) // 4, dtype=np.uint64)
    lo = np.uint64(0xFFFFFFFF)
    c = philox([j & lo, j >> np.uint64(32), np.full_like(j, offset & 0xFFFFFFFF), np.full_like(j, offset >> 32)],
               (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack(c, 1).reshape(-1)[start - 4 * first:][:n]


def factors(shape, p, rng, site, start=0):
    """0 where a value is dropped, 1 / (1 - p) elsewhere, as float64."""
    n = int(np.prod(shape))
    p = float(np.float32(p))
    if p == 0.0:
        return torch.ones(shape, dtype=torch.float64)
    keep = words(rng, site, start, n) >= np.uint64(int(p * 2 ** 32))
    return torch.from_numpy(keep.reshape(shape).astype(np.float64) / (1.0 - p))


def add(x, residual, f):
    """h and its bound: the product, the factor's own rounding and the sum."""
    d = torch.where(f != 0, x.double() * f, torch.zeros((), dtype=torch.float64, device=f.device))
    h = d if residual is None else d + residual.double()
    return h, E * (3 * d.abs() + h.abs())


def norm(h, weight, bias, kind, eps):
    """A dict: y, mean, rstd, xh, and bounds, of h as it is stored."""
    h = h.double()
    n = h.shape[-1]
    mean = h.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(h[..., :1])
    v = h - mean
    ma = v.abs().mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((v * v).sum(-1, keepdim=True) / n + eps)
    w = torch.ones(n, dtype=torch.float64, device=h.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    xh = v * rstd
    y = xh * w + b
    # the mean's error: what is left of it after the second sum, and the variance's 40 e, halved
    # by the root, with the root's and the quotient's own
    ev = E * (4 * v.abs() + 48 * ma) if kind == "layer" else torch.zeros_like(v)
    yb = rstd * w.abs() * ev + E * (48 * (xh * w).abs() + 3 * y.abs())
    mb = E * (3 * mean.abs() + 60 * ma)
    return dict(y=y, y_bound=yb, mean=mean[..., 0], mean_bound=mb[..., 0], rstd=rstd[..., 0],
                rstd_bound=48 * E * rstd[..., 0], xh=xh, w=w, v=v, mb=mb, rs=rstd)


def norm_bwd(h, dy, dh, weight, kind, eps, f):
    """Gradients by the formula, from the 64-bit mean and rstd."""
    s = norm(h, weight, None, kind, eps)
    dy = dy.double()
    xh, rs, w = s["xh"], s["rs"], s["w"]
    bx = rs * (s["mb"] + 4 * E * s["v"].abs()) + 52 * E * xh.abs()
    dn = dy * w
    s1 = dn.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(rs)
    s2 = (dn * xh).mean(-1, keepdim=True)
    e1 = 42 * E * dn.abs().mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(rs)
    e2 = (dn.abs() * bx).mean(-1, keepdim=True) + 44 * E * (dn * xh).abs().mean(-1, keepdim=True)
    t = dn - s1 - xh * s2
    g = rs * t
    b = rs * (e1 + xh.abs() * e2 + s2.abs() * bx + 6 * E * (dn.abs() + s1.abs() + (xh * s2).abs()))
    b = b + 52 * E * g.abs()
    if dh is not None:
        b = b + 2 * E * (dh.double().abs() + g.abs())
        g = g + dh.double()
    rows = dy.reshape(-1, dy.shape[-1]).shape[0]
    many = rows / 256 + 20  # rows a thread adds up in fp32, then those of its block
    flat = (-1, dy.shape[-1])
    out = dict(dresidual=g, dresidual_bound=b, dx=g * f, dx_bound=(b + 3 * E * g.abs()) * f,
               dweight=(dy * xh).reshape(flat).sum(0), dbias=dy.reshape(flat).sum(0))
    out["dweight_bound"] = (dy.abs() * bx + many * E * (dy * xh).abs()).reshape(flat).sum(0) + E * out["dweight"].abs()
    out["dbias_bound"] = many * E * dy.abs().reshape(flat).sum(0) + E * out["dbias"].abs()
    return out


def rotate(x, freqs, positions, mscale, interleaved, inverse=False):
    """x turned, and its bound: the cosine's and sine's 8 e and the angle's own rounding in 64 bits."""
    B, L, _, _ = x.shape
    n = freqs.numel()
    pos = torch.arange(L, device=x.device).expand(B, L) if positions is None else positions
    angle = pos.double()[:, :, None, None] * freqs.double()
    cos, sin = torch.cos(angle) * mscale, torch.sin(angle) * mscale * (-1 if inverse else 1)
    d = x.double()
    a, b = (d[..., 0:2 * n:2], d[..., 1:2 * n:2]) if interleaved else (d[..., :n], d[..., n:2 * n])
    y, bound = d.clone(), torch.zeros_like(d)
    off = mscale * (a.abs() + b.abs()) * (12 * E + angle.abs() * 2.0 ** -50)
    for where, v in ((0, a * cos - b * sin), (1, b * cos + a * sin)):
        if interleaved:
            y[..., where:2 * n:2], bound[..., where:2 * n:2] = v, off
        else:
            y[..., where * n:(where + 1) * n], bound[..., where * n:(where + 1) * n] = v, off
    return y, bound
