"""Dropout on the GPU: the mask of the published generator, values, residuals, gradients."""
import pytest
import torch

import layer_ref as ref
import selective_state_space_66_amd as ssm
from gated_scan_ref import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def draw(n, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn((n,), generator=gen, device=DEV).to(dtype)


@pytest.mark.parametrize("p", [0.0, 1e-9, 0.1, 0.5, 0.999])
@pytest.mark.parametrize("xt,rt", [(F32, None), (BF16, None), (F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("n", [1, 3, 8, 13, 2048, 2049, 70001])
def test_values(n, xt, rt, p):
    print(f"[dropout] {n} {xt} {rt} {p}", flush=True)
    x, res = draw(n, xt, 1), None if rt is None else draw(n, rt, 2)
    rng = torch.tensor([-3, (1 << 62) + 5], device=DEV)  # a seed with all its bits
    y = ssm.dropout_fwd(x, p, rng, site=11, residual=res)
    f = ref.factors((n,), p, rng, 11).to(DEV)
    want, bound = ref.add(x, res, f)
    check("y", y, want, bound, y.dtype)
    if res is None:
        assert torch.equal(y == 0, (f == 0) | (x == 0))
    dy = draw(n, y.dtype, 3)
    dx = ssm.dropout_bwd(dy, p, rng, site=11, dtype=xt)
    want, bound = ref.add(dy, None, f)
    assert dx.dtype == xt
    check("dx", dx, want, bound, xt)


def test_rates():
    """Of a million values as many are dropped as were asked for, within five deviations."""
    x = torch.ones(1 << 20, device=DEV)
    for p in (0.01, 0.3, 0.9):
        rng = torch.tensor([5, 6], device=DEV)
        zeros = [(ssm.dropout_fwd(x, p, rng, site=s) == 0) for s in (0, 1)]
        for z in zeros:
            assert abs(int(z.sum()) - p * 2 ** 20) <= 5 * (p * (1 - p) * 2 ** 20) ** 0.5
        both = int((zeros[0] & zeros[1]).sum())  # another site is another mask
        assert abs(both - p * p * 2 ** 20) <= 5 * (p * p * 2 ** 20) ** 0.5 + 5


def test_a_dropped_value_is_zero_whatever_it_is():
    x = draw(1000, F32, 4)
    rng = torch.tensor([7, 8], device=DEV)
    f = ref.factors((1000,), 0.4, rng, 0).to(DEV)
    x[f == 0] = float("nan")
    y = ssm.dropout_fwd(x, 0.4, rng)
    assert torch.isfinite(y).all() and not y[f == 0].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place_and_between_words(dtype):
    """Over x, over the residual, and tensors at any element: the same bits."""
    n = 5003
    x, res = draw(n, dtype, 5), draw(n, dtype, 6)
    rng = torch.tensor([9, 10], device=DEV)
    want = ssm.dropout_fwd(x, 0.2, rng, residual=res)
    for over in ("x", "res"):
        a, b = x.clone(), res.clone()
        got = ssm.dropout_fwd(a, 0.2, rng, residual=b, y=a if over == "x" else b)
        assert torch.equal(got, want)
    room = torch.empty(3 * n + 3, dtype=dtype, device=DEV)
    a, b, c = room[1:1 + n], room[n + 1:2 * n + 1], room[2 * n + 1:3 * n + 1]
    a.copy_(x)
    b.copy_(res)
    assert torch.equal(ssm.dropout_fwd(a, 0.2, rng, residual=b, y=c), want)


def test_offsets_past_32_bits():
    n = (1 << 32) + 1000
    x = torch.ones(n, dtype=BF16, device=DEV)
    rng = torch.tensor([11, 12], device=DEV)
    y = ssm.dropout_fwd(x, 0.5, rng)
    for start in (0, (1 << 32) - 500, n - 600):
        f = ref.factors((600,), 0.5, rng, 0, start=start).to(DEV)
        assert torch.equal(y[start:start + 600].double(), f)


def test_a_captured_graph_draws_anew():
    x = draw(4096, BF16, 7)
    rng = torch.tensor([13, 0], device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ssm.dropout_fwd(x, 0.3, rng)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ssm.dropout_fwd(x, 0.3, rng)
        rng[1:] += 1
    seen = []
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = ssm.dropout_fwd(x, 0.3, torch.tensor([13, step], device=DEV))
        assert torch.equal(y, want)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])


def test_refusals():
    x, rng = draw(8, F32, 8), torch.tensor([1, 2], device=DEV)
    for bad in (dict(p=1.0, rng=rng), dict(p=-0.1, rng=rng), dict(p=float("nan"), rng=rng),
                dict(p=0.5, rng=None), dict(p=0.5, rng=rng[:1]), dict(p=0.5, rng=rng.cpu())):
        with pytest.raises(ValueError):
            ssm.dropout_fwd(x, **bad)
    with pytest.raises(TypeError):
        ssm.dropout_fwd(x, 0.5, rng.int())
    with pytest.raises(TypeError):
        ssm.dropout_fwd(x, 0.5, rng, residual=x.bfloat16())
    with pytest.raises(ValueError):
        ssm.dropout_fwd(x, 0.5, rng, residual=draw(9, F32, 9))
    with pytest.raises(ValueError):
        ssm.dropout_fwd(x.view(2, 4).t(), 0.5, rng)
    assert ssm.dropout_fwd(x[:0], 0.5, rng).numel() == 0
