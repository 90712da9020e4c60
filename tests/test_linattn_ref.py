"""The 64-bit reference of linear attention against central differences of its own
forward, every input, with shared keys, lengths and document starts (CPU)."""
import numpy as np
import pytest

import linattn_ref as R


@pytest.mark.parametrize("ragged", [False, True])
def test_gradients_against_differences(ragged):
    x = R.inputs(3, 2, 9, 4, 2, 3, 5, "f32", strong=True)
    x = {k: v.astype(np.float64) for k, v in x.items()}
    lens = np.array([9, 6]) if ragged else None
    reset = np.zeros((2, 9), dtype=np.uint8)
    reset[0, 4] = reset[1, 0] = reset[1, 3] = 1
    reset = reset if ragged else None
    scale = 0.37

    def loss(y):
        o, last = R.forward(y["q"], y["k"], y["v"], y["g"], scale, y["h0"], lens, reset)
        return float((o * x["do"]).sum() + (last * x["dlast"]).sum())

    got = R.backward(x["q"], x["k"], x["v"], x["g"], x["do"], scale, x["h0"], x["dlast"], lens, reset)
    rng = np.random.default_rng(4)
    eps = 1e-5
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("h0", "dh0")):
        flat = got[key].reshape(-1)
        for i in rng.permutation(flat.size)[:40]:
            y = {k: v.copy() for k, v in x.items()}
            y[name].reshape(-1)[i] += eps
            up = loss(y)
            y[name].reshape(-1)[i] -= 2 * eps
            d = (up - loss(y)) / (2 * eps)
            # differences of a smooth function: error eps^2 in the step, 1e-16 / eps in rounding
            assert abs(d - flat[i]) <= 1e-6 * (1 + np.abs(flat).max()), (name, i, d, flat[i])


def test_one_token_at_a_time():
    x = R.inputs(5, 1, 7, 2, 1, 4, 6, "f32")
    o, last = R.forward(x["q"], x["k"], x["v"], x["g"], 1.0, x["h0"])
    S = x["h0"]
    for t in range(7):
        s = slice(t, t + 1)
        ot, S = R.forward(x["q"][:, s], x["k"][:, s], x["v"][:, s], x["g"], 1.0, S)
        assert np.allclose(ot[:, 0], o[:, t], rtol=1e-12)
    assert np.allclose(S, last, rtol=1e-12)
