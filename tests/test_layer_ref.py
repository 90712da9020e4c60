"""The 64-bit references of tests/layer_ref.py: the generator's published vectors, gradients
against differences, and the frequencies of rotary_freqs (no GPU)."""
import math

import numpy as np
import pytest
import torch

import layer_ref as ref
import selective_state_space_66_amd as ssm


@pytest.mark.parametrize("counter,key,want", [
    ([0, 0, 0, 0], [0, 0], "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ([0xffffffff] * 4, [0xffffffff] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     "d16cfe09 94fdcceb 5001e420 24126ea1")])
def test_published_vectors(counter, key, want):
    got = ref.philox([np.array([w], dtype=np.uint64) for w in counter], key)
    assert " ".join(f"{int(w[0]):08x}" for w in got) == want


def test_words_do_not_depend_on_where_one_starts():
    rng = torch.tensor([123456789012345, 987654321098765])
    whole = ref.words(rng, 7, 0, 50)
    for start in (1, 4, 13):
        assert (ref.words(rng, 7, start, 20) == whole[start:start + 20]).all()
    moved = torch.tensor([123456789012345, 987654321098765 + 7])
    assert (ref.words(moved, 0, 0, 50) == whole).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradients_against_differences(kind):
    gen = torch.Generator().manual_seed(3)
    h, dy, dh = (torch.randn((3, 6), generator=gen, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(6, generator=gen, dtype=torch.float64) for _ in range(2))
    g = ref.norm_bwd(h, dy, dh, w, kind, 1e-5, torch.ones_like(h))

    def loss(h, w, b):
        return float((ref.norm(h, w, b, kind, 1e-5)["y"] * dy).sum() + (h * dh).sum())

    for name, t, got in (("h", h, g["dresidual"]), ("w", w, g["dweight"]), ("b", b, g["dbias"])):
        for e in range(t.numel()):
            vals = []
            for sign in (1, -1):
                m = t.clone()
                m.view(-1)[e] += sign * 1e-5
                vals.append(loss(*(m if n == name else v for n, v in (("h", h), ("w", w), ("b", b)))))
            want = (vals[0] - vals[1]) / 2e-5
            assert abs(float(got.reshape(-1)[e]) - want) <= 1e-7 * (1 + abs(want)), (name, e)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_turns_back(interleaved):
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((2, 5, 3, 10), generator=gen, dtype=torch.float64)
    freqs = torch.tensor([1.0, 0.3, 0.01])
    y, _ = ref.rotate(x, freqs, None, 1.0, interleaved)
    back, _ = ref.rotate(y, freqs, None, 1.0, interleaved, inverse=True)
    assert torch.allclose(back, x, atol=1e-14) and torch.equal(y[..., 6:], x[..., 6:])
    assert torch.allclose(y.square().sum(-1), x.square().sum(-1), atol=1e-12)
    # scores depend on the distance alone
    q = x[:, :1].expand(2, 5, 3, 10)
    s = (ref.rotate(q, freqs, None, 1.0, interleaved)[0][:, 1:] * ref.rotate(q, freqs, None, 1.0, interleaved)[0][:, :-1]).sum(-1)
    assert torch.allclose(s, s[:, :1].expand_as(s), atol=1e-12)


def test_frequencies():
    f, m = ssm.rotary_freqs(8, device="cpu")
    assert m == 1.0 and f.dtype == torch.float32
    assert torch.equal(f, torch.tensor([1.0, 0.1, 0.01, 0.001]))
    f, m = ssm.rotary_freqs(8, scaling="linear", factor=4.0, device="cpu")
    assert m == 1.0 and torch.allclose(f, torch.tensor([0.25, 0.025, 0.0025, 0.00025]))
    f, _ = ssm.rotary_freqs(8, scaling="ntk", factor=4.0, device="cpu")
    assert f[0] == 1.0 and math.isclose(float(f[3]), 0.001 / 4.0, rel_tol=1e-6)
    f, m = ssm.rotary_freqs(64, scaling="yarn", factor=8.0, original_length=4096, device="cpu")
    base, _ = ssm.rotary_freqs(64, device="cpu")
    assert math.isclose(m, 1.0 + 0.1 * math.log(8.0))
    turns = 4096 * base / (2 * math.pi)
    assert torch.equal(f[turns > 40], base[turns > 40])
    assert torch.allclose(f[turns < 0.7], base[turns < 0.7] / 8.0)
    ratio = f / base
    assert (ratio[1:] <= ratio[:-1] * (1 + 1e-6)).all()  # the ramp falls
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="other"),
                dict(rot_dim=8, factor=0.5), dict(rot_dim=8, theta=1.0), dict(rot_dim=8, scaling="yarn")):
        with pytest.raises(ValueError):
            ssm.rotary_freqs(**bad, device="cpu")
