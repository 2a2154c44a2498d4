"""GPU parity of the rotary position encoding with the fp64 oracle.

Bound: the angle is a 64-bit product reduced to a turn and rounded to fp32 (at most
pi 2^-24 absolute), cos and sin are within 2 ulp, then two products and a sum in
fp32: 12 * 2^-24 of (|x| + |x'|) * scale, and one rounding to the type."""

import numpy as np
import pytest
import torch

from gated_delta_rule_82_amd import kda
from oracle import attn_oracle as ora
from tests.attn_check import BF16, F32, U, U24, check, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    kda.load()
    yield
    torch.cuda.synchronize()


def want(x, pos, f, scale, il, inv):
    ref = ora.rotary(np64(x), np64(pos), f, scale, il, inv)
    mass = ora.rotary(np.abs(np64(x)), np.zeros(pos.shape), f, abs(scale), il)  # |x| in the first of a pair, |x'| in the second
    rot = 2 * len(f)
    first = np.arange(0, rot, 2) if il else np.arange(rot // 2)
    second = first + 1 if il else first + rot // 2
    pair = mass[..., first] + mass[..., second]
    mass[..., first], mass[..., second] = pair, pair
    return ref, 12 * U24 * mass + U[x.dtype] * (np.abs(ref) + 12 * U24 * mass)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,rot", [(16, 16), (16, 2), (32, 24), (64, 32), (64, 6), (128, 128), (128, 96), (128, 126)])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("B,T,H,HK", [(1, 1, 1, 1), (3, 17, 5, 2), (2, 130, 4, 0)])
def test_rotary_matches_oracle(dtype, D, rot, il, B, T, H, HK):
    g = torch.Generator().manual_seed(D + rot + T)
    x = torch.randn(B, T, H + HK + 1, D, generator=g).to(dtype).cuda()   # one more head that stays as it is
    before = x.clone()
    q, k = x[:, :, :H], x[:, :, H:H + HK] if HK else None
    pos = torch.randint(-50, 1 << 20, (B, T), generator=g, dtype=torch.int32)
    for scaling, inv in (("none", False), ("yarn", True)):
        f, s = kda.rotary_freqs(rot, scaling=scaling, factor=4.0, trained=4096)
        fr, sr = ora.rotary_freqs(rot, scaling=scaling, factor=4.0, trained=4096)
        assert np.allclose(np64(f), fr, rtol=1e-14, atol=0) and abs(s - sr) < 1e-7
        out = kda.rotary(q, k, f, pos.cuda(), scale=s, interleaved=il, inverse=inv)
        torch.cuda.synchronize()
        for y, xin in zip((out,) if k is None else out, (q, k)):
            check(y, *want(xin, pos, np64(f), s, il, inv), "rotary")
        assert torch.equal(x, before)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rot", [64, 20])
def test_rotary_in_place_on_a_packed_projection(dtype, rot):
    x = torch.randn(2, 9, 4 + 2 + 2, 64, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    f, _ = kda.rotary_freqs(rot)
    q, k = x[:, :, :4], x[:, :, 4:6]
    a, b = kda.rotary(q, k, f)
    y = x.clone()
    kda.rotary(y[:, :, :4], y[:, :, 4:6], f, q_out=y[:, :, :4], k_out=y[:, :, 4:6])
    torch.cuda.synchronize()
    assert torch.equal(y[:, :, :4], a) and torch.equal(y[:, :, 4:6], b) and torch.equal(y[:, :, 6:], x[:, :, 6:])
    pos = torch.arange(9, dtype=torch.int32, device="cuda").expand(2, 9).contiguous()
    for u, w in zip(kda.rotary(q, k, f, pos), (a, b)):
        assert torch.equal(u, w)


def test_rotary_inverse_is_the_transpose():
    g = torch.Generator().manual_seed(4)
    x, y = (torch.randn(2, 33, 3, 128, generator=g).cuda() for _ in range(2))
    f, s = kda.rotary_freqs(96, scaling="yarn", factor=8.0, trained=2048)
    pos = torch.randint(0, 100000, (2, 33), generator=g, dtype=torch.int32).cuda()
    for il in (False, True):
        fx = kda.rotary(x, None, f, pos, scale=s, interleaved=il)
        ty = kda.rotary(y, None, f, pos, scale=s, interleaved=il, inverse=True)
        a, b = float((np64(fx) * np64(y)).sum()), float((np64(x) * np64(ty)).sum())
        # each side's elements are off by at most 12 * 2^-24 of a pair's magnitude, 1.21 = scale bound
        tol = 2 * 12 * U24 * 1.3 * 2 * float((np.abs(np64(x)) + 1).sum() + (np.abs(np64(y)) + 1).sum()) * 4
        assert abs(a - b) < tol


def test_rotary_empty_and_refusals():
    f, _ = kda.rotary_freqs(16)
    q = torch.randn(0, 4, 2, 32, device="cuda")
    assert kda.rotary(q, None, f).shape == (0, 4, 2, 32)
    q = torch.randn(2, 4, 2, 32, device="cuda")
    with pytest.raises(TypeError):
        kda.rotary(q.half(), None, f)
    with pytest.raises(TypeError):
        kda.rotary(q, None, f.float())
    with pytest.raises(ValueError):
        kda.rotary(q, None, f, torch.zeros(4, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kda.rotary(q.transpose(1, 2), None, f)
    with pytest.raises(ValueError):
        kda.rotary(q.cpu(), None, f.cpu())
    with pytest.raises(kda.KDAError):
        kda.rotary(q, None, kda.rotary_freqs(64)[0])                         # more channels than a head has
    with pytest.raises(kda.KDAError):
        kda.rotary(q, None, f, scale=float("nan"))
    buf = torch.randn(2, 5, 2, 32, device="cuda")
    with pytest.raises(kda.KDAError):
        kda.rotary(buf.view(-1)[:256].view(1, 4, 2, 32), None, f, q_out=buf.view(-1)[64:320].view(1, 4, 2, 32))
