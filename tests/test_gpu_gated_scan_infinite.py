"""Infinite states of the gated linear recurrence: a_t is more than 0, so a state that is infinite stays
infinite, of its sign, to its document's end, in calls of either type and of any length."""
import pytest
import torch

import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def inputs(B, L, dim, io, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    d = {n: torch.randn((B, L, dim), generator=gen, device=DEV).to(io) for n in ("x", "r", "i")}
    # forgetting little (1 - a is what is kept) and much
    d["decay"] = torch.linspace(1e-3, 4.0, dim, device=DEV)
    return d, torch.randn((B, dim), generator=gen, device=DEV), gen


# one token, a wave's and a chunk's share, many chunks, groups of chunks
SIZES = [(2, 1, 6), (2, 5, 6), (2, 64, 70), (2, 128, 6), (2, 700, 66), (1, 9000, 40)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("B,L,dim", SIZES)
def test_an_infinite_state_stays(B, L, dim, io):
    print(f"[gated scan] infinite {B} x {L} x {dim} {io}", flush=True)
    d, h0, gen = inputs(B, L, dim, io, 1)
    clean = ssm.gated_scan_fwd(**d, h0=h0)
    start = h0.clone()
    start[:, 0], start[:, 1] = INF, -INF  # from before the first token
    where = L // 3
    d["x"][:, where, 2], d["x"][:, where, 3] = INF, -INF  # from a token on
    y, last, _ = ssm.gated_scan_fwd(**d, h0=start)
    assert (y[:, :, 0] == INF).all() and (y[:, :, 1] == -INF).all()
    assert (y[:, where:, 2] == INF).all() and (y[:, where:, 3] == -INF).all()
    for c, want in enumerate((INF, -INF, INF, -INF)):
        assert (last[:, c] == want).all()
    # nothing else changes
    assert torch.equal(y[:, :, 4:], clean[0][:, :, 4:]) and torch.equal(last[:, 4:], clean[1][:, 4:])
    assert torch.equal(y[:, :where, 2:4], clean[0][:, :where, 2:4])
    if L >= 64:  # up to where a document starts
        reset = torch.zeros((B, L), dtype=torch.bool, device=DEV)
        reset[:, where + 20] = True
        cut, last, _ = ssm.gated_scan_fwd(**d, h0=start, reset=reset)
        assert (cut[:, :where + 20, 0] == INF).all() and (cut[:, where:where + 20, 3] == -INF).all()
        assert torch.isfinite(cut[:, where + 20:]).all() and torch.isfinite(last).all()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("B,L,dim", SIZES)
def test_an_infinite_gradient_stays(B, L, dim, io):
    """The gradient of the state goes through the same factors from the end."""
    d, h0, gen = inputs(B, L, dim, io, 2)
    dy = torch.randn((B, L, dim), generator=gen, device=DEV).to(io)
    dlast = torch.randn((B, dim), generator=gen, device=DEV)
    states = ssm.gated_scan_fwd(**d, h0=h0, return_states=True)[2]
    clean = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True)
    where = L // 3
    dlast[:, 0], dlast[:, 1] = INF, -INF
    dy[:, where, 2], dy[:, where, 3] = INF, -INF
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True)
    for c, want in enumerate((INF, -INF, INF, -INF)):
        assert (g["dh0"][:, c] == want).all()
        assert (g["dx"][:, :where + 1, c] == want).all()  # times the root and the gate, both more than 0
    assert (g["dx"][:, :, 0] == INF).all() and (g["dx"][:, :, 1] == -INF).all()
    assert torch.equal(g["dx"][:, where + 1:, 2:4], clean["dx"][:, where + 1:, 2:4])
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][..., 4:], clean[n][..., 4:])
    assert torch.equal(g["ddecay"][4:], clean["ddecay"][4:])


@pytest.mark.parametrize("io", [F32, BF16])
def test_an_infinite_state_stays_in_steps(io):
    d, h0, _ = inputs(3, 9, 6, io, 3)
    state = h0.clone()
    state[:, 0], state[:, 1] = INF, -INF
    d["x"][:, 4, 2], d["x"][:, 4, 3] = INF, -INF
    for t in range(9):
        y = ssm.gated_scan_step(state, *(d[n][:, t].contiguous() for n in ("x", "r", "i")), d["decay"])
        assert torch.equal(y, state.to(io)) and torch.isfinite(state[:, 4:]).all()
        assert (state[:, 0] == INF).all() and (state[:, 1] == -INF).all()
        assert (state[:, 2] == INF).all() == (t >= 4) and (state[:, 3] == -INF).all() == (t >= 4)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("L", [64, 128, 700, 9000])
def test_the_largest_finite_state_is_forgotten(L, io):
    """A state of 3e38 that nothing is left of after a while: less than 2^-149 of it is, so no more
    than 3e38 2^-149 = 4e-7 stays where a factor is held in 32 bits, and that is forgotten too."""
    d, h0, gen = inputs(2, L, 6, io, 4)
    d["decay"].fill_(12.0)
    d["r"] = d["r"].abs()  # v of 6 and more: 2^-149 after 18 tokens
    h0[:, 0], h0[:, 1] = 3e38, -3e38
    clean = ssm.gated_scan_fwd(**d, h0=torch.zeros_like(h0))
    y, last, _ = ssm.gated_scan_fwd(**d, h0=h0)
    for got, want in ((y[:, 20:], clean[0][:, 20:]), (last, clean[1])):
        err = (got.double() - want.double()).abs()
        # each side's rounding to its type, and sums of a few terms in another order
        assert (err <= 1e-6 + (torch.finfo(got.dtype).eps + 16 * 2.0 ** -24) * want.double().abs()).all()
    assert torch.equal(y[:, 64:], clean[0][:, 64:])
