"""The gated linear recurrence at the ends of its sizes and values."""
import pytest
import torch

import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(0, 4, 5), (2, 0, 5), (0, 0, 5), (0, 700, 5)])
def test_without_tokens_the_decay_has_no_gradient(shape, io):
    """Zero, where the decay is 0 too."""
    z = torch.zeros(shape, dtype=io, device=DEV)
    decay = torch.tensor([0.0, 1.0, 0.0, 1e-3, 2.0], device=DEV)
    _, last, states = ssm.gated_scan_fwd(z, z, z, decay, return_states=True)
    ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device=DEV)
    g = ssm.gated_scan_bwd(z, z, z, decay, z, states, dlast=last, workspace=ws)
    assert torch.equal(g["ddecay"], torch.zeros(5, device=DEV))


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [40, 700])
def test_the_largest_decay(L, io):
    """Of 1e30 nothing is kept: y is the gated input, gradients go through that alone."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, r, i, dy = (torch.randn((2, L, 70), generator=gen, device=DEV).to(io) for _ in range(4))
    h0, dlast = (torch.randn((2, 70), generator=gen, device=DEV) for _ in range(2))
    decay = torch.full((70,), 1e30, device=DEV)
    y, last, states = ssm.gated_scan_fwd(x, r, i, decay, h0=h0, return_states=True)
    g = ssm.gated_scan_bwd(x, r, i, decay, dy, states, dlast=dlast, need_dh0=True)
    gate = torch.sigmoid(i.double())
    lam = dy.double()
    lam[:, -1] += dlast.double()
    # a sigmoid (12 e: its argument is below 6), its rest and three products or sums, then the type's rounding
    tol = 32 * 2.0 ** -24 + torch.finfo(io).eps / 2
    for got, want in ((y, gate * x.double()), (g["dx"], lam * gate), (g["di"], lam * x.double() * gate * (1 - gate))):
        assert ((got.double() - want).abs() <= tol * want.abs()).all()
    assert torch.equal(last.to(io), y[:, -1])
    for n in ("dr", "ddecay", "dh0"):
        assert torch.isfinite(g[n]).all() and g[n].abs().max() <= 1e-7, n
