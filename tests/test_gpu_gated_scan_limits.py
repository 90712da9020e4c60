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


def test_more_blocks_than_one_dimension_of_a_grid():
    """4.2 million rows of one channel: past 2^32 threads the blocks have a second number.  One token (a
    block of 1024 threads a row), and two chunks a row, whose blocks also take numbers and wait."""
    for B, L in ((4_200_000, 1), (4_200_000, 130)):
        print(f"[gated scan] {B} x {L} x 1", flush=True)
        x, r, i, dy = (torch.zeros((B, L, 1), dtype=torch.bfloat16, device=DEV) for _ in range(4))
        gen = torch.Generator(device=DEV).manual_seed(L)
        rows = [0, 1, 65535, 4_194_295, 4_194_296, 4_194_303, 4_194_304, B - 2, B - 1]
        few = [torch.randn((len(rows), L, 1), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(4)]
        for t, f in zip((x, r, i, dy), few):
            t[rows] = f
        h0 = torch.full((B, 1), 0.5, device=DEV)
        decay = torch.tensor([0.3], device=DEV)
        y, last, states = ssm.gated_scan_fwd(x, r, i, decay, h0=h0, return_states=True)
        alone = ssm.gated_scan_fwd(*few[:3], decay, h0=h0[:len(rows)], return_states=True)
        for got, want in zip((y, last, states), alone):
            assert torch.equal(got[rows], want)
        g = ssm.gated_scan_bwd(x, r, i, decay, dy, states, dlast=h0, need_dh0=True)
        want = ssm.gated_scan_bwd(*few[:3], decay, few[3], alone[2], dlast=h0[:len(rows)], need_dh0=True)
        for n in ("dx", "dr", "di", "dh0"):
            assert torch.equal(g[n][rows], want[n]), n
        # all the other rows have the same inputs, and so the same outputs
        rest = torch.ones(B, dtype=torch.bool, device=DEV)
        rest[rows] = False
        for t in (y, last, g["dh0"], g["dr"]):
            assert (t[rest] == t[2]).all()


def test_a_nan_and_the_gradients_around_it():
    """A NaN in a token reaches the gradients of its document from there on through the state (dr) and to
    its start through the adjoint (all of them), and nothing of another document."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    d = {n: torch.randn((1, 500, 70), generator=gen, device=DEV) for n in ("x", "r", "i")}
    d["decay"] = torch.rand((70,), generator=gen, device=DEV) + 1e-3
    dy = torch.randn((1, 500, 70), generator=gen, device=DEV)
    reset = torch.zeros((1, 500), dtype=torch.bool, device=DEV)
    reset[0, [131, 300]] = True
    states = ssm.gated_scan_fwd(**d, reset=reset, return_states=True)[2]
    clean = ssm.gated_scan_bwd(**d, dy=dy, states=states, reset=reset)
    for n in ("x", "r", "i"):
        d[n][0, 140:142] = float("nan")
    states = ssm.gated_scan_fwd(**d, reset=reset, return_states=True)[2]
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, reset=reset)
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][0, :131], clean[n][0, :131]) and torch.equal(g[n][0, 300:], clean[n][0, 300:]), n
        assert torch.isnan(g[n][0, 131:142]).all(), n
    assert torch.isnan(g["dr"][0, 142:300]).all()  # of a state that is a NaN
    assert torch.equal(g["dx"][0, 142:300], clean["dx"][0, 142:300])
    assert torch.equal(g["di"][0, 142:300], clean["di"][0, 142:300])
    assert torch.isnan(g["ddecay"]).all()
