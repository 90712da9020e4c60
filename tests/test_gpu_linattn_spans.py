"""Linear attention over axes long enough that the walks run in several spans, each after the
states of finer pieces before it, for the tiles of all head sizes: with shared keys, a length
and documents that end inside a piece, against dense products in 64 bits.  Workspaces hold NaN
before the first call and what it left before the second, and both give the same bits.

Bounds as for the short sequences (1e-5 for fp32 results, 4e-3 for bf16 ones).  The log-decay's
gradient is a sum over tokens that may cancel: its error is measured against the larger of the
result and the root of its terms' squares.
"""
import numpy as np
import pytest
import torch

import linattn_ref as R
import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = {torch.float32: 1e-5, torch.bfloat16: 4e-3}


def dense(q, k, v, g, scale, h0, do, dlast, n, starts):
    """One head of one entry: n real tokens; starts: the flags of document starts.  All float64.
    Returns o, last, dq, dk, dv, dh0 and the tokens' terms of dg (the state's one last)."""
    L = q.shape[0]
    t = torch.arange(L, device=DEV)
    seg = torch.cumsum(torch.where(t < n, starts, torch.zeros_like(starts)), 0)
    live = t < n
    see = (t[:, None] >= t[None, :]) & (seg[:, None] == seg[None, :]) & live[:, None] & live[None, :]
    dist = (t[:, None] - t[None, :]).double()
    w = torch.where(see, torch.exp(g * dist.clamp(min=0)), torch.zeros((), device=DEV).double())
    # the initial state at each token, every token's part in the last state
    w0 = torch.where(live & (seg == 0), torch.exp(g * (t + 1).double()), torch.zeros((), device=DEV).double())
    ends = seg[n - 1] if n else 0
    w1 = torch.where(live & (seg == ends), torch.exp(g * (n - 1 - t).double().clamp(min=0)), torch.zeros((), device=DEV).double())
    e0 = torch.exp(g * n) * float(ends == 0)
    s, r = q @ k.T, do @ v.T
    o = scale * ((s * w) @ v + w0[:, None] * (q @ h0.T))
    last = (v * w1[:, None]).T @ k + e0 * h0
    out = dict(o=o, last=last)
    out["dq"] = scale * ((r * w) @ k + w0[:, None] * (do @ h0))
    out["dk"] = scale * ((r * w).T @ q) + w1[:, None] * (v @ dlast)
    out["dv"] = scale * ((s * w).T @ do) + w1[:, None] * (k @ dlast.T)
    out["dh0"] = scale * ((do * w0[:, None]).T @ q) + e0 * dlast
    terms = scale * ((s * r * w * dist).sum(1) + w0 * (t + 1) * ((do @ h0) * q).sum(1))
    final = (w1 * (n - 1 - t) * ((v @ dlast) * k).sum(1)).sum() + e0 * n * (dlast * h0).sum()
    out["dg"] = torch.cat([terms, final[None]])
    return out


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("H,Dk,Dv", [(8, 32, 32), (8, 64, 40), (8, 128, 32), (6, 72, 96), (8, 40, 128),
                                     (8, 128, 128), (4, 256, 64), (4, 64, 256), (4, 136, 200)])
def test_spans(H, Dk, Dv, ragged, io):
    B, Hk, L, scale = 2, H // 2, 4033, 0.2
    print(f"[linattn] spans H{H}/{Hk} D{Dk}x{Dv} {io} ragged={ragged}", flush=True)
    rng = np.random.default_rng(Dk + Dv)

    def draw(*shape):
        return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(DEV)

    q, k, v, do = (draw(B, L, n, d).to(io) for n, d in ((Hk, Dk), (Hk, Dk), (H, Dv), (H, Dv)))
    h0, dlast = draw(B, H, Dv, Dk), draw(B, H, Dv, Dk)
    g = torch.from_numpy(np.log1p(-np.exp2(-np.linspace(4.0, 10.0, H))).astype(np.float32)).to(DEV)
    lens, reset = [L, L], torch.zeros((B, L), dtype=torch.uint8, device=DEV)
    if ragged:
        lens = [L, 2345]
        for b, t in ((0, 700), (0, 2100), (0, 3999), (1, 64), (1, 1000), (1, 1001), (1, 3000)):
            reset[b, t] = 1
    kw = dict(scale=scale, h0=h0, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV) if ragged else None,
              reset=reset if ragged else None)
    sizes = (B, L, H, Hk, Dk, Dv, io)
    assert ssm.linattn_fwd_workspace_size(*sizes) > 0
    need = max(ssm.linattn_fwd_workspace_size(*sizes), ssm.linattn_bwd_workspace_size(*sizes))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    runs = []
    for _ in range(2):
        o, last = ssm.linattn_fwd(q, k, v, g, workspace=ws, **kw)
        got = ssm.linattn_bwd(q, k, v, g, do, dlast=dlast, workspace=ws, **kw)
        got.update(o=o, last=last)
        alone = ssm.linattn_bwd(q, k, v, g, do, dlast=dlast, workspace=ws, need_dlog_decay=False, **kw)
        got.update({n + " alone": alone[n] for n in ("dq", "dk", "dv", "dh0")})
        runs.append(got)
    torch.cuda.synchronize()
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n
    got = runs[0]
    assert alone["dlog_decay"] is None

    d = {n: t.double() for n, t in dict(q=q, k=k, v=v, do=do, h0=h0, dlast=dlast, g=g).items()}
    want = dict(o=torch.zeros_like(d["v"]), dv=torch.zeros_like(d["v"]), dq=torch.zeros_like(d["q"]),
                dk=torch.zeros_like(d["k"]), last=torch.zeros_like(d["h0"]), dh0=torch.zeros_like(d["h0"]))
    dg = torch.zeros((H, B * (L + 1)), device=DEV).double()
    for b in range(B):
        for h in range(H):
            i = h // (H // Hk)
            x = dense(d["q"][b, :, i], d["k"][b, :, i], d["v"][b, :, h], d["g"][h], scale, d["h0"][b, h],
                      d["do"][b, :, h], d["dlast"][b, h], lens[b], reset[b].long())
            want["o"][b, :, h], want["dv"][b, :, h] = x["o"], x["dv"]
            want["dq"][b, :, i] += x["dq"]
            want["dk"][b, :, i] += x["dk"]
            want["last"][b, h], want["dh0"][b, h] = x["last"], x["dh0"]
            dg[h, b * (L + 1):(b + 1) * (L + 1)] = x["dg"]
    for n in ("o", "dq", "dk", "dv", "last", "dh0", "dq alone", "dk alone", "dv alone", "dh0 alone"):
        ref = want[n.split()[0]]
        tol = 1e-5 if n.split()[0] in ("last", "dh0") else TOL[io]
        assert got[n].shape == ref.shape and torch.isfinite(got[n]).all(), n
        err = float((got[n].double() - ref).norm() / ref.norm())
        assert err <= tol, f"{n}: {err:.2e}"
    total = dg.sum(1)
    size = torch.maximum(total.abs(), dg.square().sum(1).sqrt())
    err = float((got["dlog_decay"].double() - total).norm() / size.norm())
    assert err <= 1e-5, f"dlog_decay: {err:.2e}"


def test_dense_reference():
    """The dense form against the token by token one."""
    x = {n: a.astype(np.float64) for n, a in R.inputs(40, 1, 50, 1, 1, 8, 8, "f32", strong=True).items()}
    t = {n: torch.from_numpy(a).to(DEV) for n, a in x.items()}
    reset = np.zeros((1, 50), dtype=np.uint8)
    reset[0, [0, 20, 45]] = 1
    for lens, r in ((50, None), (33, reset), (1, reset), (50, reset)):
        flags = torch.from_numpy(reset[0] if r is not None else np.zeros(50, dtype=np.uint8)).to(DEV).long()
        y = dense(t["q"][0, :, 0], t["k"][0, :, 0], t["v"][0, :, 0], t["g"][0], 0.3, t["h0"][0, 0],
                  t["do"][0, :, 0], t["dlast"][0, 0], lens, flags)
        o, last = R.forward(x["q"], x["k"], x["v"], x["g"], 0.3, x["h0"], np.array([lens]), r)
        g = R.backward(x["q"], x["k"], x["v"], x["g"], x["do"], 0.3, x["h0"], x["dlast"], np.array([lens]), r)
        for n, ref in (("o", o[0, :, 0]), ("last", last[0, 0]), ("dq", g["dq"][0, :, 0]), ("dk", g["dk"][0, :, 0]),
                       ("dv", g["dv"][0, :, 0]), ("dh0", g["dh0"][0, 0])):
            assert np.allclose(y[n].cpu().numpy(), ref, rtol=1e-9, atol=1e-9), n
        assert abs(float(y["dg"].sum()) - g["dlog_decay"][0]) <= 1e-9 * max(1.0, abs(g["dlog_decay"][0]))
