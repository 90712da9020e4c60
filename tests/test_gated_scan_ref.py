"""The 64-bit reference of the gated linear recurrence against central differences (no GPU)."""
import pytest
import torch

import gated_scan_ref as ref


@pytest.mark.parametrize("masked", [False, True])
def test_gradients_against_differences(masked):
    gen = torch.Generator().manual_seed(5)
    B, L, dim = 2, 9, 3

    def normal(*shape):
        return torch.randn(shape, generator=gen, dtype=torch.float64)

    x, r, i, dy = (normal(B, L, dim) for _ in range(4))
    decay = torch.tensor([1e-3, 0.3, 2.5], dtype=torch.float64)
    h0, dlast = normal(B, dim), normal(B, dim)
    lens = torch.tensor([L, 5]) if masked else None
    reset = torch.zeros((B, L), dtype=torch.uint8)
    reset[0, 4] = reset[1, 0] = 1
    reset = reset if masked else None
    kw = dict(seq_lens=lens, reset=reset)

    def loss(x, r, i, decay, h0):
        f = ref.forward(x, r, i, decay, h0=h0, **kw)
        return float((f["y"] * dy).sum() + (f["last_state"] * dlast).sum())

    g = ref.backward(x, r, i, decay, dy, dlast=dlast, h0=h0, **kw)
    args = dict(x=x, r=r, i=i, decay=decay, h0=h0)
    for name in args:
        t = args[name]
        for e in range(t.numel()):
            step = 1e-6 if name == "decay" else 1e-5
            vals = []
            for sign in (1, -1):
                moved = t.clone()
                moved.view(-1)[e] += sign * step
                vals.append(loss(**{**args, name: moved}))
            want = (vals[0] - vals[1]) / (2 * step)
            got = float(g["d" + name].reshape(-1)[e])
            # the differences' own rounding, 1e-15 of a sum of some 50 terms over the step, and
            # their third-order term (decay's is step^2 / decay^3 of the value)
            assert abs(got - want) <= 1e-7 + 1e-5 * abs(want), (name, e, got, want)


def test_padding_is_truncation_and_reset_is_a_new_sequence():
    gen = torch.Generator().manual_seed(6)
    x, r, i = (torch.randn((1, 8, 2), generator=gen, dtype=torch.float64) for _ in range(3))
    decay = torch.tensor([0.1, 1.0])
    whole = ref.forward(x, r, i, decay, seq_lens=torch.tensor([5]))
    short = ref.forward(x[:, :5], r[:, :5], i[:, :5], decay)
    assert torch.equal(whole["y"][:, :5], short["y"]) and not whole["y"][:, 5:].any()
    assert torch.equal(whole["last_state"], short["last_state"])
    flags = torch.zeros((1, 8), dtype=torch.uint8)
    flags[0, 3] = 1
    cut = ref.forward(x, r, i, decay, reset=flags)
    assert torch.equal(cut["y"][:, 3:], ref.forward(x[:, 3:], r[:, 3:], i[:, 3:], decay)["y"])
