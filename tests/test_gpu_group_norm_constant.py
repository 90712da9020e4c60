"""Group norm of values that hardly vary beside a large common offset, one row per entry.

A constant group: mean exact to fp32, variance zero, so rstd = eps^-1/2 and y = bias.  What is
left of x - mean is its rounding: the mean is held in two parts, each a sum of at most 32 values
in a lane and 6 across lanes, times 1 / count, so off by at most 40 * 2^-24 of what it sums: 1600
* 2^-48 = 5.7e-12 of the offset, times rstd in y.  The variance is that squared, beside eps.
"""
import pytest
import torch

import selective_state_space_66_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("cg", [1, 3, 7, 24, 64, 100, 200, 255, 256])
@pytest.mark.parametrize("offset,eps", [(3.0, 1e-5), (1e3, 1e-8), (1e5, 1e-12), (-1e5, 1e-12), (1e8, 1e-6)])
def test_constant_groups(cg, offset, eps):
    groups, n = 3, 64
    gen = torch.Generator(device=DEV).manual_seed(cg)
    values = offset * (1 + torch.rand((n, groups), generator=gen, device=DEV))
    x = values.repeat_interleave(cg, 1).view(n, 1, groups * cg).contiguous()
    bias = torch.arange(groups * cg, dtype=torch.float32, device=DEV)
    y, mean, rstd = ssm.group_norm_fwd(x, groups, bias=bias, eps=eps)
    dx = ssm.group_norm_bwd(x, groups, torch.ones_like(x), mean, rstd, bias=bias)["dx"]
    torch.cuda.synchronize()
    print(f"[group norm] constant {offset} cg {cg} eps {eps}", flush=True)
    left = 5.7e-12 * 2 * abs(offset)
    want = (left * left + eps) ** -0.5, eps ** -0.5
    assert torch.isfinite(rstd).all() and torch.isfinite(y).all() and torch.isfinite(dx).all()
    assert (rstd >= want[0] * (1 - 3e-7)).all() and (rstd <= want[1] * (1 + 3e-7)).all()
    assert ((mean - values).abs() <= 2.0 ** -24 * values.abs()).all()
    # the bias, rounded once more, and what is left of x - mean
    assert ((y[:, 0] - bias).abs() <= left * want[1] + 2.0 ** -23 * bias).all()


@pytest.mark.parametrize("cg", [24, 64, 100, 256])
def test_small_variation(cg):
    """Values a few units in the last place about an offset: the variance of exactly those."""
    gen = torch.Generator(device=DEV).manual_seed(cg)
    x = 65536.0 + torch.randint(0, 5, (64, 1, 2 * cg), generator=gen, device=DEV).float() / 128
    y, mean, rstd = ssm.group_norm_fwd(x, 2, eps=1e-8)
    xs = x.double().view(64, 2, cg)
    mu = xs.mean(2, keepdim=True)
    rs = ((xs - mu).square().mean(2, keepdim=True) + 1e-8).rsqrt()
    want = ((xs - mu) * rs).view(64, 1, -1)
    assert float((rstd.double() - rs[..., 0]).norm() / rs.norm()) <= 1e-5
    assert float((y.double() - want).norm() / want.norm()) <= 1e-5
