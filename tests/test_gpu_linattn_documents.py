"""What a document holds stays in it: NaN and infinities at its last tokens, or at the first
tokens of the next one, reach no output of a chunk of 64 tokens that holds none of them, no
state, and change no bit there (within a chunk the products take all of its tokens)."""
import numpy as np
import pytest
import torch

import linattn_ref as R
import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def run(x, io, reset):
    t = {n: torch.from_numpy(x[n]).to(DEV).to(io) for n in ("q", "k", "v", "do")}
    g, h0, dlast = (torch.from_numpy(x[n]).to(DEV) for n in ("g", "h0", "dlast"))
    o, last = ssm.linattn_fwd(t["q"], t["k"], t["v"], g, h0=h0, reset=reset)
    grads = ssm.linattn_bwd(t["q"], t["k"], t["v"], g, t["do"], h0=h0, dlast=dlast, reset=reset)
    plain = ssm.linattn_bwd(t["q"], t["k"], t["v"], g, t["do"], h0=h0, dlast=dlast, reset=reset,
                            need_dlog_decay=False)
    out = dict(o=o, last=last, dh0=grads["dh0"])
    for n in ("dq", "dk", "dv"):
        out[n], out[n + " alone"] = grads[n], plain[n]
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,start,Dk,Dv", [(200, 100, 64, 64), (200, 100, 128, 64), (200, 127, 72, 128),
                                           (200, 65, 256, 40), (200, 101, 40, 256), (2100, 1060, 64, 40),
                                           (2100, 1060, 128, 128)])
def test_other_documents(L, start, Dk, Dv, io):
    print(f"[linattn] documents L{L} start {start} D{Dk}x{Dv} {io}", flush=True)
    x = R.inputs(800 + Dk + Dv, 1, L, 2, 1, Dk, Dv, "f32" if io == torch.float32 else "bf16")
    reset = torch.zeros((1, L), dtype=torch.uint8, device=DEV)
    reset[0, start] = 1
    clean = run(x, io, reset)
    lo, hi = start // 64 * 64, (start // 64 + 1) * 64  # the chunk where one document ends
    for at, after in ((start - 1, True), (start, False)):
        for name in ("q", "k", "v", "do"):
            bad = {n: a.copy() for n, a in x.items()}
            bad[name][0, at, :, ::3] = np.nan
            bad[name][0, at, :, 1::3] = np.inf
            got = run(bad, io, reset)
            for n in got:
                if n == "last":
                    a, b = (got[n], clean[n]) if after else (None, None)
                elif n == "dh0":
                    a, b = (None, None) if after else (got[n], clean[n])
                else:  # the other document's chunks that do not hold the token
                    part = slice(hi, None) if after else slice(0, lo)
                    a, b = got[n][:, part], clean[n][:, part]
                if a is not None:
                    assert torch.isfinite(a.float()).all() and torch.equal(a, b), (name, after, n)
