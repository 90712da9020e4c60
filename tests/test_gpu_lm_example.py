"""The example that trains and serves a linear-attention layer, run as a user runs it: its
loss falls, its gradients are clipped to the norm, and token by token it computes what a
prompt of the same tokens does."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_linear_attention as example  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_trains_and_serves(io):
    model, losses, norms = example.train(steps=40, io=io)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}", flush=True)
    assert losses[-1] < 0.7 * losses[0]
    assert all(n > 0 and n < 1e3 for n in norms)
    total = sum(float(p.grad.double().square().sum()) for p in model.parameters()) ** 0.5
    assert total <= 1.0 + 1e-5  # the last step's gradients, as clipped
    generator = torch.Generator(device="cuda:0")
    generator.manual_seed(5)
    prompt = example.batch(generator, 3, 50, 32, "cuda:0")
    tokens, seen = example.generate(model, prompt, 20)
    with torch.no_grad():
        whole = model(torch.cat([prompt, tokens], 1))[:, 49:69]
    err = float((seen - whole).norm() / whole.norm())
    # one rounding of q, k, v, the gate and the two outputs to bf16 on each path (2^-8), or fp32
    assert err <= (2 * 2.0 ** -8 if io == torch.bfloat16 else 1e-4), err
