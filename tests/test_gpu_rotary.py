"""Rotary positions on the GPU against 64 bits: layouts, parts of a head, far positions,
gradients, in place."""
import pytest
import torch

import layer_ref as ref
import selective_state_space_66_amd as ssm
from gated_scan_ref import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def make(B, L, H, Hk, D, io, seed=1):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn((B, L, h, D), generator=gen, device=DEV).to(io) for h in (H, Hk)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,L,H,Hk,D,rot", [
    (1, 1, 1, 1, 2, 2), (2, 5, 3, 1, 7, 4), (1, 9, 2, 2, 16, 16), (2, 33, 4, 4, 40, 10),
    (2, 70, 6, 2, 64, 64), (2, 21, 3, 2, 40, 20), (1, 50, 9, 4, 96, 24), (2, 6, 2, 1, 36, 12), (1, 300, 8, 1, 96, 48), (3, 65, 5, 5, 128, 32), (64, 1, 24, 8, 128, 128),
    (1, 130, 2, 2, 256, 254), (2, 40, 1, 0, 64, 32)])
def test_forward_and_gradient(B, L, H, Hk, D, rot, interleaved, io):
    print(f"[rotary] {B} x {L} x {H}/{Hk} x {D} rot {rot} {interleaved} {io}", flush=True)
    q, k = make(B, L, H, Hk, D, io)
    freqs, _ = ssm.rotary_freqs(rot, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(2)
    far = torch.randint(0, 1 << 20, (B, L), generator=gen, device=DEV).to(torch.int32)
    for positions, mscale in ((None, 1.0), (far, 1.25)):
        kw = dict(positions=positions, mscale=mscale, interleaved=interleaved)
        for fn, back in ((ssm.rotary_fwd, False), (ssm.rotary_bwd, True)):
            qo, ko = fn(q, k if Hk else None, freqs, **kw)
            for name, x, got in (("q", q, qo), ("k", k, ko)):
                if got is None:
                    assert Hk == 0
                    continue
                want, bound = ref.rotate(x, freqs, positions, mscale, interleaved, back)
                check(name, got, want, bound, io)
                assert torch.equal(got[..., rot:], x[..., rot:])
        # in place: the same bits
        a, b = q.clone(), k.clone()
        ssm.rotary_fwd(a, b if Hk else None, freqs, q_out=a, k_out=b if Hk else None, **kw)
        qo, ko = ssm.rotary_fwd(q, k if Hk else None, freqs, **kw)
        assert torch.equal(a, qo) and (ko is None or torch.equal(b, ko))


def test_the_largest_and_negative_positions():
    q, k = make(1, 6, 2, 1, 64, F32)
    freqs, _ = ssm.rotary_freqs(64, device=DEV)
    pos = torch.tensor([[0, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 1_000_003]], device=DEV).to(torch.int32)
    qo, ko = ssm.rotary_fwd(q, k, freqs, positions=pos)
    for x, got in ((q, qo), (k, ko)):
        want, bound = ref.rotate(x, freqs, pos, 1.0, False)
        check("far", got, want, bound)


def test_tensors_between_words():
    q, k = make(2, 11, 3, 2, 64, BF16)
    freqs, _ = ssm.rotary_freqs(32, device=DEV)

    def shifted(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        room[1:] = t.reshape(-1)
        return room[1:].view(t.shape)

    for interleaved in (False, True):
        want = ssm.rotary_fwd(q, k, freqs, interleaved=interleaved)
        got = ssm.rotary_fwd(shifted(q), shifted(k), freqs, interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("D,rot", [(64, 32), (36, 12), (40, 20), (11, 8), (9, 2)])
def test_what_is_copied_is_copied_bit_by_bit(D, rot, io):
    """Signalling NaNs and subnormal values too, and with the queries in place alone."""
    bits = torch.int32 if io == F32 else torch.int16
    gen = torch.Generator(device=DEV).manual_seed(3)
    info = torch.iinfo(bits)
    q, k = make(2, 37, 5, 2, D, io)
    for t in (q, k):
        t[..., rot:] = torch.randint(info.min, info.max, t[..., rot:].shape, generator=gen, device=DEV,
                                     dtype=bits).view(io)
    q[0, 0, :, rot:] = torch.tensor(1, dtype=bits, device=DEV).view(io)
    freqs, _ = ssm.rotary_freqs(rot, device=DEV)
    for interleaved in (False, True):
        a = q.clone()
        qo, ko = ssm.rotary_fwd(q, k, freqs, interleaved=interleaved)
        _, kb = ssm.rotary_fwd(a, k, freqs, interleaved=interleaved, q_out=a)
        for got, x in ((qo, q), (ko, k), (a, q), (kb, k)):
            assert torch.equal(got[..., rot:].contiguous().view(bits), x[..., rot:].contiguous().view(bits))
        assert torch.equal(a[..., :rot], qo[..., :rot]) and torch.equal(kb[..., :rot], ko[..., :rot])


def test_offsets_past_32_bits():
    L, H, D = 1 << 20, 33, 128
    q = torch.zeros((1, L, H, D), dtype=BF16, device=DEV)
    tail, k = make(1, 5, H, 2, D, BF16)
    q[:, -5:] = tail
    freqs, _ = ssm.rotary_freqs(D, device=DEV)
    out = ssm.rotary_fwd(q, None, freqs)[0]
    pos = torch.arange(L - 5, L, device=DEV)[None].to(torch.int32)
    want, bound = ref.rotate(tail, freqs, pos, 1.0, False)
    check("tail", out[:, -5:], want, bound, BF16)
    assert not out[:, :-5].any()


def test_empty_and_refused():
    q, k = make(1, 4, 2, 1, 16, F32)
    freqs, _ = ssm.rotary_freqs(16, device=DEV)
    assert ssm.rotary_fwd(q[:, :0], k[:, :0], freqs)[0].shape == (1, 0, 2, 16)
    for bad in (dict(freqs=torch.ones(9, device=DEV)), dict(freqs=torch.ones(0, device=DEV)),
                dict(positions=torch.zeros((1, 3), dtype=torch.int32, device=DEV)), dict(k=k[:, :3]),
                dict(k=k[..., :8].contiguous())):
        with pytest.raises(ValueError):
            ssm.rotary_fwd(**{**dict(q=q, k=k, freqs=freqs), **bad})
    with pytest.raises(TypeError):
        ssm.rotary_fwd(q, k.bfloat16(), freqs)
    with pytest.raises(TypeError):
        ssm.rotary_fwd(q, k, freqs, positions=torch.zeros((1, 4), dtype=torch.int64, device=DEV))
