"""Gradients of gates that are nearly open or shut: what is left of a gate to 1, or the gate itself, is
2e-9 there and still a bf16 number, so dr and di have their relative accuracy.

What the bounds of gated_scan_ref have to hold, by the kernels' chunks and groups: ddecay's partial
sums add the 8 tokens of a thread and 8 waves (calls of 64 tokens at most: 4 and 16), 20 roundings at
most of the 24 it counts.  A state passes up to 31 joins before a block in a group of 32 chunks and one
with the group's state: these cover 31 chunks of 64 tokens and more, for each token of which the bound
adds 5.5 e, so that a join of 5.5 e is less than one token's share of a chunk.  The joins inside a block
(8 waves, 16 in short calls) and its first state are in the 64 e it adds once."""
import pytest
import torch

import gated_scan_ref as ref
import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# one chunk, many chunks, and (bf16) two channels a thread
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,dim", [(2, 33, 66), (2, 300, 96), (7, 1000, 981)])
def test_gradients(B, L, dim, io):
    print(f"[gated scan] open gates {B} x {L} x {dim} {io}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    ends = torch.tensor([8.0, -8.0, 12.0, -12.0, 16.0, -16.0, 20.0, -20.0, 0.0, 1.0], device=DEV)
    d = dict(x=normal(B, L, dim).to(TYPES[io]))
    for n in ("r", "i"):
        pick = torch.randint(0, ends.numel(), (B, L, dim), generator=gen, device=DEV)
        d[n] = ends[pick].to(TYPES[io])
    d["decay"] = 1e-3 * 2000.0 ** torch.rand((dim,), generator=gen, device=DEV)
    h0, dy, dlast = normal(B, dim), normal(B, L, dim).to(TYPES[io]), normal(B, dim)
    states = ssm.gated_scan_fwd(**d, h0=h0, return_states=True)[2]
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True)
    want = ref.backward(**d, dy=dy, dlast=dlast, h0=h0)
    for n in ("dx", "dr", "di"):
        ref.check(n, g[n], want[n], want[n + "_bound"], TYPES[io])
    for n in ("dh0", "ddecay"):
        ref.check(n, g[n], want[n], want[n + "_bound"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_nan_in_a_gate_is_one_in_its_gradients(io):
    gen = torch.Generator(device=DEV).manual_seed(2)
    d = {n: torch.randn((1, 200, 8), generator=gen, device=DEV).to(TYPES[io]) for n in ("x", "r", "i")}
    d["decay"] = torch.rand((8,), generator=gen, device=DEV)
    dy = torch.randn((1, 200, 8), generator=gen, device=DEV).to(TYPES[io])
    d["r"][0, 150, 1] = d["i"][0, 150, 3] = float("nan")
    states = ssm.gated_scan_fwd(**d, return_states=True)[2]
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states)
    assert torch.isnan(g["dx"][0, 150, 3]) and torch.isnan(g["di"][0, 150, 3])
    assert torch.isnan(g["dx"][0, 150, 1]) and torch.isnan(g["dr"][0, 150, 1])
    for n in ("dx", "dr", "di"):
        assert torch.isfinite(g[n][..., [0, 2, 4, 5, 6, 7]]).all()
