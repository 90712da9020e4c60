"""Linear attention with a decay for each head in 64 bits, token by token, on the CPU:
the definition the GPU tests compare with.

    S_t = lam S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t,  lam = e^g
    G_t = scale do_t q_t^T + lam G_{t+1},  dq_t = scale S_t^T do_t,  dk_t = G_t^T v_t,
    dv_t = G_t k_t,  dg = sum_t lam <G_t, S_{t-1}>
"""
import numpy as np


def forward(q, k, v, g, scale, h0=None, seq_lens=None, reset=None, keep_states=False):
    B, L, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    rep = H // Hk
    o = np.zeros((B, L, H, Dv))
    last = np.zeros((B, H, Dv, Dk)) if h0 is None else np.array(h0, dtype=np.float64)
    states = {}
    lam = np.exp(np.asarray(g, dtype=np.float64))
    for b in range(B):
        n = L if seq_lens is None else min(max(int(seq_lens[b]), 0), L)
        for h in range(H):
            S = last[b, h]
            for t in range(n):
                before = S * (0.0 if reset is not None and reset[b, t] else 1.0)
                S = lam[h] * before + np.outer(v[b, t, h], k[b, t, h // rep])
                o[b, t, h] = scale * S @ q[b, t, h // rep]
                if keep_states:
                    states[b, h, t] = (before, S)
            last[b, h] = S
    return (o, last, states) if keep_states else (o, last)


def backward(q, k, v, g, do, scale, h0=None, dlast=None, seq_lens=None, reset=None):
    B, L, Hk, Dk = q.shape
    H, Dv = v.shape[2:]
    rep = H // Hk
    _, _, states = forward(q, k, v, g, scale, h0, seq_lens, reset, keep_states=True)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg = np.zeros(H)
    dh0 = np.zeros((B, H, Dv, Dk))
    lam = np.exp(np.asarray(g, dtype=np.float64))
    for b in range(B):
        n = L if seq_lens is None else min(max(int(seq_lens[b]), 0), L)
        for h in range(H):
            kh = h // rep
            G = np.zeros((Dv, Dk)) if dlast is None else np.array(dlast[b, h], dtype=np.float64)
            for t in range(n - 1, -1, -1):
                before, S = states[b, h, t]
                G = G + scale * np.outer(do[b, t, h], q[b, t, kh])
                dq[b, t, kh] += scale * S.T @ do[b, t, h]
                dk[b, t, kh] += G.T @ v[b, t, h]
                dv[b, t, h] = G @ k[b, t, kh]
                dg[h] += lam[h] * np.sum(G * before)
                G = lam[h] * G * (0.0 if reset is not None and reset[b, t] else 1.0)
            dh0[b, h] = G
    return dict(dq=dq, dk=dk, dv=dv, dlog_decay=dg, dh0=dh0)


def inputs(seed, B, L, H, Hk, Dk, Dv, io, strong=False):
    """float32 arrays whose values bf16 holds exactly where io is "bf16"."""
    rng = np.random.default_rng(seed)

    def draw(*shape):
        x = rng.normal(size=shape).astype(np.float32)
        if io == "bf16":  # round to nearest even at 8 bits
            u = x.view(np.uint32).astype(np.uint64)
            x = ((u + 0x7fff + ((u >> 16) & 1)) & 0xffff0000).astype(np.uint32).view(np.float32)
        return x

    e = np.linspace(0.5, 4.0, H) if strong else np.linspace(4.0, 10.0, H)
    return dict(q=draw(B, L, Hk, Dk), k=draw(B, L, Hk, Dk), v=draw(B, L, H, Dv),
                do=draw(B, L, H, Dv), g=np.log1p(-np.exp2(-e)).astype(np.float32),
                h0=rng.normal(size=(B, H, Dv, Dk)).astype(np.float32),
                dlast=rng.normal(size=(B, H, Dv, Dk)).astype(np.float32))
