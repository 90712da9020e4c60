"""The gated linear recurrence on the GPU against its 64-bit reference: sequences, gradients,
one token, at the sizes where waves, chunks and groups of chunks meet."""
import pytest
import torch

import gated_scan_ref as ref
import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, L, dim, io, seed, masked, slowest=1e-3):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    d = dict(x=normal(B, L, dim).to(io), r=normal(B, L, dim).to(io), i=normal(B, L, dim).to(io))
    u = torch.rand((dim,), generator=gen, device=DEV)
    d["decay"] = slowest * (2.0 / slowest) ** u
    kw = dict(seq_lens=None, reset=None)
    if masked:
        kw["seq_lens"] = torch.randint(0, L + 1, (B,), generator=gen, device=DEV).to(torch.int32)
        kw["seq_lens"][-1] = L
        if B > 1:
            kw["seq_lens"][0] = 0  # a row with no token
        kw["reset"] = torch.rand((B, L), generator=gen, device=DEV) < 3.0 / L
    return d, normal(B, dim), normal(B, L, dim).to(io), normal(B, dim), kw


# one token, a wave's share and one past it, a chunk and one past it, a group of 32 chunks and
# one past it, three groups; channels that fill no tile, odd ones, one tile and one past it
SIZES = [(1, 1, 1), (2, 7, 3), (1, 17, 66), (1, 33, 64), (3, 128, 130), (2, 129, 66), (1, 257, 65),
         (2, 300, 128), (2, 640, 192), (1, 4096, 10), (1, 4097, 8), (2, 9000, 70)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,L,dim", SIZES)
def test_forward(B, L, dim, masked, io):
    print(f"[gated scan] forward {B} x {L} x {dim} {io} masked {masked}", flush=True)
    d, h0, _, _, kw = inputs(B, L, dim, TYPES[io], 1, masked)
    for start in (None, h0):
        y, last, states = ssm.gated_scan_fwd(**d, h0=start, return_states=True, **kw)
        torch.cuda.synchronize()
        want = ref.forward(**d, h0=start, **kw)
        ref.check("y", y, want["y"], want["y_bound"], TYPES[io])
        ref.check("last_state", last, want["last_state"], want["last_bound"])
        ref.check("states", states, want["before"][:, ::64], want["before_bound"][:, ::64] + 1e-36)
        assert not y[~want["live"]].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,L,dim", SIZES)
def test_backward(B, L, dim, masked, io):
    print(f"[gated scan] backward {B} x {L} x {dim} {io} masked {masked}", flush=True)
    d, h0, dy, dlast, kw = inputs(B, L, dim, TYPES[io], 2, masked)
    states = ssm.gated_scan_fwd(**d, h0=h0, return_states=True, **kw)[2]
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True, **kw)
    torch.cuda.synchronize()
    want = ref.backward(**d, dy=dy, dlast=dlast, h0=h0, **kw)
    for n in ("dx", "dr", "di"):
        ref.check(n, g[n], want[n], want[n + "_bound"], TYPES[io])
    for n in ("dh0", "ddecay"):
        ref.check(n, g[n], want[n], want[n + "_bound"])
    # without what is optional: the same bits in the rest
    less = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_ddecay=False, **kw)
    assert less["ddecay"] is None and less["dh0"] is None
    for n in ("dx", "dr", "di"):
        assert torch.equal(less[n], g[n])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1e-6, 20.0, 300.0])
def test_decays_at_the_ends_of_their_range(decay, io):
    """Nothing forgotten (and nothing taken in), memories of a million tokens, and of none."""
    print(f"[gated scan] decay {decay} {io}", flush=True)
    d, h0, dy, dlast, kw = inputs(2, 700, 96, TYPES[io], 3, False)
    d["decay"].fill_(decay)
    y, last, states = ssm.gated_scan_fwd(**d, h0=h0, return_states=True)
    want = ref.forward(**d, h0=h0)
    ref.check("y", y, want["y"], want["y_bound"], TYPES[io])
    ref.check("last_state", last, want["last_state"], want["last_bound"])
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True)
    if decay == 0.0:
        assert torch.equal(last, h0) and not g["dx"].any() and not g["dr"].any()
        return
    want = ref.backward(**d, dy=dy, dlast=dlast, h0=h0)
    for n in ("dx", "dr", "di", "dh0", "ddecay"):
        ref.check(n, g[n], want[n], want[n + "_bound"], TYPES[io] if n in ("dx", "dr", "di") else torch.float32)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gates_far_out(io):
    """Gates at +-30, +-100 and infinity are open or shut, with finite gradients."""
    d, h0, dy, dlast, kw = inputs(1, 160, 64, TYPES[io], 4, False)
    ends = torch.tensor([30.0, -30.0, 100.0, -100.0, float("inf"), -float("inf")], device=DEV).to(TYPES[io])
    d["r"][0, 3:9], d["i"][0, 20:26] = ends[:, None], ends[:, None]
    y, last, states = ssm.gated_scan_fwd(**d, return_states=True)
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states)
    for t in (y, last, g["dx"], g["dr"], g["di"], g["ddecay"]):
        assert torch.isfinite(t).all()
    big = {n: t.float().clamp(-80, 80).to(t.dtype) if n in "ri" else t for n, t in d.items()}
    want = ref.forward(**big)
    # sigmoid(80) and sigmoid(inf) are one number in 32 bits, sigmoid(-80) is 2e-35: a state of
    # up to 4 moves by v of 4e-35 at most, an input by the root of it, 1e-17
    ref.check("y", y, want["y"], want["y_bound"] + 1e-16, TYPES[io])


def test_padding_and_documents_hold_a_nan_back():
    """NaN past a length and in another document reach nothing else."""
    d, h0, dy, dlast, kw = inputs(2, 500, 70, torch.float32, 5, False)
    lens = torch.tensor([200, 500], dtype=torch.int32, device=DEV)
    reset = torch.zeros((2, 500), dtype=torch.bool, device=DEV)
    reset[1, [131, 300]] = True
    clean = ssm.gated_scan_fwd(**d, seq_lens=lens, reset=reset, return_states=True)
    gc = ssm.gated_scan_bwd(**d, dy=dy, states=clean[2], seq_lens=lens, reset=reset)
    for n in ("x", "r", "i"):
        d[n][0, 200:] = float("nan")
        d[n][1, 140:142] = float("nan")
    dy[0, 200:] = float("nan")
    h0[1] = float("nan")  # before the first document of the second row
    y, last, states = ssm.gated_scan_fwd(**d, h0=h0 * torch.tensor([[0.0], [1.0]], device=DEV),
                                         seq_lens=lens, reset=reset, return_states=True)
    assert torch.equal(y[0], clean[0][0]) and torch.equal(y[1, 300:], clean[0][1, 300:])
    assert torch.equal(last, clean[1])
    assert torch.isnan(y[1, :131]).all() and torch.isnan(y[1, 140:300]).all()
    assert torch.equal(y[1, 131:140], clean[0][1, 131:140])
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, seq_lens=lens, reset=reset)
    for n in ("dx", "dr", "di"):
        assert torch.equal(g[n][0], gc[n][0]) and torch.equal(g[n][1, 300:], gc[n][1, 300:])
        assert torch.equal(g[n][1, 142:300].isnan(), torch.zeros_like(g[n][1, 142:300]).bool() if n != "dr"
                           else g[n][1, 142:300].isnan())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("every", [1, 7, 64, 128, 512])
def test_documents_side_by_side(every, io):
    """A document starts at every token, between waves, at chunks and at groups of chunks; each is
    a sequence of its own, whatever the state before it."""
    L = 1300
    d, h0, dy, dlast, _ = inputs(2, L, 66, TYPES[io], 13, False)
    reset = torch.zeros((2, L), dtype=torch.uint8, device=DEV)
    reset[:, ::every] = 1
    h0.fill_(float("nan"))
    y, last, states = ssm.gated_scan_fwd(**d, h0=h0, reset=reset, return_states=True)
    want = ref.forward(**d, reset=reset)
    ref.check("y", y, want["y"], want["y_bound"], TYPES[io])
    ref.check("last_state", last, want["last_state"], want["last_bound"])
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, reset=reset, need_dh0=True)
    want = ref.backward(**d, dy=dy, dlast=dlast, reset=reset)
    for n in ("dx", "dr", "di"):
        ref.check(n, g[n], want[n], want[n + "_bound"], TYPES[io])
    ref.check("ddecay", g["ddecay"], want["ddecay"], want["ddecay_bound"])
    assert not g["dh0"].any()


@pytest.mark.parametrize("rows,dim", [(1, 100), (1, 200), (1, 700), (1, 1500), (2, 1030), (3, 1100)])
def test_groups_of_every_size(rows, dim):
    """Rows for groups of 32, 16, 8 and 4 chunks, forwards and backwards, a few groups long."""
    d, h0, dy, dlast, kw = inputs(rows, 4500, dim, torch.bfloat16, 14, True)
    y, last, states = ssm.gated_scan_fwd(**d, h0=h0, return_states=True, **kw)
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True, **kw)
    torch.cuda.synchronize()
    want = ref.backward(**d, dy=dy, dlast=dlast, h0=h0, **kw)
    f = ref.forward(**d, h0=h0, **kw)
    ref.check("y", y, f["y"], f["y_bound"], torch.bfloat16)
    ref.check("last_state", last, f["last_state"], f["last_bound"])
    for n in ("dx", "dr", "di"):
        ref.check(n, g[n], want[n], want[n + "_bound"], torch.bfloat16)
    for n in ("dh0", "ddecay"):
        ref.check(n, g[n], want[n], want[n + "_bound"])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_steps_make_the_sequence(io):
    d, h0, _, _, _ = inputs(3, 40, 130, TYPES[io], 6, False)
    y, last, _ = ssm.gated_scan_fwd(**d, h0=h0)
    want = ref.forward(**d, h0=h0)
    state = h0.clone()
    for t in range(40):
        out = ssm.gated_scan_step(state, d["x"][:, t].contiguous(), d["r"][:, t].contiguous(),
                                  d["i"][:, t].contiguous(), d["decay"])
        ref.check(f"y {t}", out, want["y"][:, t], want["y_bound"][:, t], TYPES[io])
    ref.check("state", state, want["last_state"], want["last_bound"])


@pytest.mark.parametrize("dim", [1, 3, 64, 5120])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_sizes(dim, io):
    for B in (1, 5):
        d, h0, _, _, _ = inputs(B, 1, dim, TYPES[io], 7, False)
        state = h0.clone()
        flat = {n: d[n][:, 0].contiguous() for n in ("x", "r", "i")}
        y = ssm.gated_scan_step(state, decay=d["decay"], **flat)
        want = ref.forward(**d, h0=h0)
        ref.check("y", y, want["y"][:, 0], want["y_bound"][:, 0], TYPES[io])
        ref.check("state", state, want["last_state"], want["last_bound"])
        again = ssm.gated_scan_step(h0, decay=d["decay"], y=flat["x"], **flat)  # over its input
        assert again is flat["x"] and torch.equal(again, y)


def test_tensors_that_start_between_words():
    """bf16 tensors aligned to two bytes give the bits of aligned ones."""
    d, h0, dy, dlast, kw = inputs(2, 300, 192, torch.bfloat16, 8, True)

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    want = ssm.gated_scan_fwd(**d, h0=h0, return_states=True, **kw)
    odd = {n: shifted(t) if n != "decay" else t for n, t in d.items()}
    got = ssm.gated_scan_fwd(**odd, h0=h0, return_states=True, y=shifted(want[0]), **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    gw = ssm.gated_scan_bwd(**d, dy=dy, states=want[2], dlast=dlast, **kw)
    gg = ssm.gated_scan_bwd(**odd, dy=shifted(dy), states=want[2], dlast=dlast, **kw)
    for n in ("dx", "dr", "di", "ddecay"):
        assert torch.equal(gg[n], gw[n])


# small ones, and bf16 of 6.3 million values and more in rows of no whole lines, which threads take
# two channels of: many chunks, and one (forwards); a last one that two tiles have
WIDE = [(3, 1100, 1999), (3, 1100, 2002), (50, 100, 1271), (7, 1000, 981), (7, 1000, 1025)]


@pytest.mark.parametrize("B,L,dim", [(2, 333, 65), (2, 333, 191), (2, 333, 1537)] + WIDE)
def test_a_last_channel_of_its_own_is_like_any_other(B, L, dim):
    """Odd rows of bf16 give the bits of rows with one more channel, and nothing behind them."""
    print(f"[gated scan] {B} x {L} x {dim} beside one more channel", flush=True)
    d, h0, dy, dlast, kw = inputs(B, L, dim + 1, torch.bfloat16, 15, True)

    def cut(t):
        return t[..., :dim].contiguous()

    def room(t):  # for an output, with a mark behind it
        flat = torch.full((t.numel() + 1,), 7.0, dtype=t.dtype, device=DEV)
        return flat, flat[:-1].view(t.shape)

    want = ssm.gated_scan_fwd(**d, h0=h0, return_states=True, **kw)
    odd = {n: cut(t) for n, t in d.items()}
    flat, y = room(odd["x"])
    got = ssm.gated_scan_fwd(**odd, h0=cut(h0), return_states=True, y=y, **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, cut(b))
    assert flat[-1] == 7.0
    gw = ssm.gated_scan_bwd(**d, dy=dy, states=want[2], dlast=dlast, need_dh0=True, **kw)
    for _ in range(3):
        gg = ssm.gated_scan_bwd(**odd, dy=cut(dy), states=got[2], dlast=cut(dlast), need_dh0=True, **kw)
        for n in gw:
            assert torch.equal(gg[n], cut(gw[n])), n


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("B,L,dim", WIDE)
def test_two_channels_a_thread(B, L, dim, masked):
    print(f"[gated scan] {B} x {L} x {dim} masked {masked}", flush=True)
    d, h0, dy, dlast, kw = inputs(B, L, dim, torch.bfloat16, 16, masked)
    y, last, states = ssm.gated_scan_fwd(**d, h0=h0, return_states=True, **kw)
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, need_dh0=True, **kw)
    torch.cuda.synchronize()
    f = ref.forward(**d, h0=h0, **kw)
    ref.check("y", y, f["y"], f["y_bound"], torch.bfloat16)
    ref.check("last_state", last, f["last_state"], f["last_bound"])
    assert not y[~f["live"]].any()
    want = ref.backward(**d, dy=dy, dlast=dlast, h0=h0, **kw)
    for n in ("dx", "dr", "di"):
        ref.check(n, g[n], want[n], want[n + "_bound"], torch.bfloat16)
        assert not g[n][~f["live"]].any()
    for n in ("dh0", "ddecay"):
        ref.check(n, g[n], want[n], want[n + "_bound"])


def test_empty_calls():
    z = torch.zeros((2, 0, 5), device=DEV)
    decay, h0 = torch.ones(5, device=DEV), torch.randn((2, 5), device=DEV)
    y, last, states = ssm.gated_scan_fwd(z, z, z, decay, h0=h0, return_states=True)
    assert y.shape == (2, 0, 5) and torch.equal(last, h0) and states.shape == (2, 0, 5)
    assert not ssm.gated_scan_fwd(z, z, z, decay)[1].any()
    g = ssm.gated_scan_bwd(z, z, z, decay, z, states, dlast=h0, need_dh0=True)
    assert torch.equal(g["dh0"], h0) and not g["ddecay"].any()
    none = torch.zeros((0, 4, 5), device=DEV)
    y, last, states = ssm.gated_scan_fwd(none, none, none, decay, return_states=True)
    assert last.shape == (0, 5)
    assert not ssm.gated_scan_bwd(none, none, none, decay, none, states)["ddecay"].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L", [0, 40, 1000])
def test_a_state_without_tokens_is_kept_as_it_is(L, io):
    """Rows of length 0 hand their state on bit for bit, an infinity and a tiny number too, and
    the gradient of the last state back."""
    d, h0, dy, dlast, _ = inputs(2, L, 8, TYPES[io], 15, False)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    h0[0] = torch.tensor([float("inf"), -float("inf"), 1e-38, 3e38, 0.0, -0.5, 1.0, 7e-20], device=DEV)
    y, last, states = ssm.gated_scan_fwd(**d, h0=h0, seq_lens=lens, return_states=True)
    assert torch.equal(last, h0) and not y.any()
    g = ssm.gated_scan_bwd(**d, dy=dy, states=states, dlast=dlast, seq_lens=lens, need_dh0=True)
    assert torch.equal(g["dh0"], dlast)
    for n in ("dx", "dr", "di", "ddecay"):
        assert not g[n].any()


def test_same_bits_again_on_another_stream_and_beside_another_call():
    a, h0, dy, dlast, kw = inputs(4, 5000, 256, torch.bfloat16, 9, True)
    b = inputs(2, 7000, 192, torch.float32, 10, False)[0]

    def run(d, **more):
        return ssm.gated_scan_fwd(**d, return_states=True, **more)

    want, other = run(a, h0=h0, **kw), run(b)
    grads = ssm.gated_scan_bwd(**a, dy=dy, states=want[2], dlast=dlast, **kw)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            p = run(a, h0=h0, **kw)
            g = ssm.gated_scan_bwd(**a, dy=dy, states=p[2], dlast=dlast, **kw)
        with torch.cuda.stream(s2):
            q = run(b)
        torch.cuda.synchronize()
        for got, expected in ((p, want), (q, other)):
            for t, w in zip(got, expected):
                assert torch.equal(t, w)
        for n in ("dx", "dr", "di", "ddecay"):
            assert torch.equal(g[n], grads[n])


def test_a_workspace_that_held_something_else():
    d, h0, dy, dlast, kw = inputs(2, 4500, 96, torch.bfloat16, 11, False)
    want = ssm.gated_scan_fwd(**d, return_states=True)
    for fill in (0, 255, 1):
        ws = torch.full((ssm.gated_scan_workspace_size(2, 4500, 96),), fill, dtype=torch.uint8, device=DEV)
        got = ssm.gated_scan_fwd(**d, return_states=True, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    """4.5 GB a tensor: the last documents of the last row, against the same tokens alone."""
    B, L, dim = 2, 1_100_000, 1024
    gen = torch.Generator(device=DEV).manual_seed(12)
    tail = 300
    d = {}
    short = {}
    for n in ("x", "r", "i"):
        short[n] = torch.randn((1, tail, dim), generator=gen, device=DEV).to(torch.bfloat16)
        d[n] = torch.zeros((B, L, dim), dtype=torch.bfloat16, device=DEV)
        d[n][-1, -tail:] = short[n][0]
    decay = torch.rand((dim,), generator=gen, device=DEV)
    reset = torch.zeros((B, L), dtype=torch.uint8, device=DEV)
    reset[-1, L - tail] = 1
    y, last, states = ssm.gated_scan_fwd(**d, decay=decay, reset=reset, return_states=True)
    want = ref.forward(**short, decay=decay)
    ref.check("y", y[-1:, -tail:], want["y"], want["y_bound"], torch.bfloat16)
    ref.check("last_state", last[-1:], want["last_state"], want["last_bound"])
    dy = torch.zeros_like(y)
    del y
    dy[-1, -tail:] = short["x"][0].flip(0)
    g = ssm.gated_scan_bwd(**d, decay=decay, dy=dy, states=states, reset=reset)
    want = ref.backward(**short, decay=decay, dy=dy[-1:, -tail:])
    for n in ("dx", "dr", "di"):
        ref.check(n, g[n][-1:, -tail:], want[n], want[n + "_bound"], torch.bfloat16)
    ref.check("ddecay", g["ddecay"], want["ddecay"], want["ddecay_bound"])
