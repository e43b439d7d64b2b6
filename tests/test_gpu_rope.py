"""Rotary positions against the 64-bit form.

Tolerance.  cos and sin are fp32 values of an angle reduced in fp64: the reduced turn in
[-1/2, 1/2] is rounded to fp32 (2^-26 turns at most, 2^-23.3 rad) and sincospif is good to a few
steps, so each is off by at most 2^-22; |y| <= mscale (|a| + |b|), the two products and the sum
round by 3 2^-24 of that.  Together 2^-21 (|a| + |b|) mscale, plus the output's half step.
"""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def limit(x, e, inv_freq, rot_begin, interleaved, mscale):
    half = inv_freq.numel()
    j = torch.arange(half)
    ia, ib = (rot_begin + 2 * j, rot_begin + 2 * j + 1) if interleaved else (rot_begin + j, rot_begin + half + j)
    t = torch.zeros(x.shape, dtype=torch.float64)
    size = (x.double()[..., ia].abs() + x.double()[..., ib].abs()) * mscale
    t[..., ia] = size * 2.0 ** -21
    t[..., ib] = size * 2.0 ** -21
    return t + e.abs() * HALF[x.dtype] + 1e-38


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,begin,rot", [(128, 0, 128), (64, 32, 32), (64, 0, 20), (80, 6, 50), (7, 1, 6), (66, 2, 64),
                                         (4, 0, 2), (8, 3, 0)])
def test_rope(crs, cuda_dev, dtype, interleaved, D, begin, rot):
    g = torch.Generator().manual_seed(D + rot)
    for n_tok, heads in ((1, 1), (37, 5), (300, 16)):
        x = torch.randn(n_tok, heads, D, generator=g).to(dtype)
        pos = torch.randint(-50, 2 ** 20, (n_tok,), generator=g).to(torch.int32)
        f = crs.rope_inv_freq(rot, base=1e4, device="cpu") if rot else torch.zeros(0, dtype=torch.float64)
        for inverse, ms in ((False, 1.0), (True, 1.3)):
            y = crs.rope(x.to(cuda_dev), pos.to(cuda_dev), f.to(cuda_dev), rot_begin=begin, interleaved=interleaved,
                         mscale=ms, inverse=inverse)
            e = ref.rope(x, pos, f, begin, interleaved, ms, inverse)
            assert ((y.double().cpu() - e).abs() <= limit(x, e, f, begin, interleaved, ms)).all()
            lo, hi = x[..., :begin], x[..., begin + rot:]                 # the rest is copied
            assert torch.equal(y[..., :begin].cpu(), lo) and torch.equal(y[..., begin + rot:].cpu(), hi)
    assert crs.get_device_error() == 0


def test_far_positions_keep_their_angle(crs, cuda_dev):
    """Positions near 2^31: an fp32 angle would be wrong by whole turns."""
    pos = torch.tensor([2 ** 31 - 1, 2 ** 30 + 12345, 2 ** 24 + 1, -2 ** 31], dtype=torch.int32)
    x = torch.randn(4, 3, 64, generator=torch.Generator().manual_seed(1))
    f = crs.rope_inv_freq(64, base=1e6, device="cpu")
    y = crs.rope(x.to(cuda_dev), pos.to(cuda_dev), f.to(cuda_dev)).double().cpu()
    e = ref.rope(x, pos, f)
    # the 64-bit reference's own angle is off by 2^31 2^-53 turns' worth on either side
    assert ((y - e).abs() <= limit(x, e, f, 0, False, 1.0) + 2.0 ** -20).all()


def test_in_place_strided_and_its_own_inverse(crs, cuda_dev):
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    qkv = torch.randn(50, 12, 64, generator=g, device=cuda_dev)
    keep = qkv.clone()
    pos = torch.arange(50, dtype=torch.int32, device=cuda_dev)
    f = crs.rope_inv_freq(64)
    q = qkv[:, 2:7]                                            # rows of 5 heads, 12 apart
    dense = crs.rope(q, pos, f)
    crs.rope(q, pos, f, out=q)
    assert torch.equal(q, dense)
    assert torch.equal(qkv[:, :2], keep[:, :2]) and torch.equal(qkv[:, 7:], keep[:, 7:])
    back = crs.rope(q, pos, f, inverse=True)
    assert (back - keep[:, 2:7]).abs().max() <= 2.0 ** -18 * keep.abs().max()
    odd = torch.randn(50 * 5 * 64 + 1, generator=g, device=cuda_dev)[1:].view(50, 5, 64)     # 4-byte aligned
    assert torch.equal(crs.rope(odd, pos, f), crs.rope(odd.clone(), pos, f))


def test_gradient(crs, cuda_dev):
    """inverse=True is the transpose: <rope(x), w> = <x, rope^T(w)>, against differences too."""
    g = torch.Generator(device=cuda_dev).manual_seed(4)
    x = torch.randn(9, 4, 64, generator=g, device=cuda_dev)
    w = torch.randn(9, 4, 64, generator=g, device=cuda_dev)
    pos = torch.randint(0, 10 ** 6, (9,), generator=g, device=cuda_dev).to(torch.int32)
    f = crs.rope_inv_freq(32, base=1e4, factor=4.0)
    kw = dict(rot_begin=16, interleaved=True, mscale=1.2)
    grad = crs.rope(w, pos, f, inverse=True, **kw).double()
    xc, wc = x.double().cpu(), w.double().cpu()
    e = torch.zeros_like(xc)                                   # the formula, entry by entry of the 64-bit form
    xr = xc.clone().requires_grad_(True)
    (ref.rope(xr, pos.cpu(), f.cpu(), 16, True, 1.2) * wc).sum().backward()
    e = xr.grad
    assert ((grad.cpu() - e).abs() <= limit(w.cpu(), e, f.cpu(), 16, True, 1.2)).all()
    h = 2.0 ** -3                                              # linear: a difference of any step is exact
    for t, hd, j in ((0, 0, 16), (3, 2, 17), (8, 3, 47), (5, 1, 0)):
        d = torch.zeros_like(x)
        d[t, hd, j] = h
        num = ((crs.rope(x + d, pos, f, **kw).double() - crs.rope(x - d, pos, f, **kw).double()) * w.double()).sum()
        assert abs(float(num) / (2 * h) - float(grad[t, hd, j])) <= 2.0 ** -16


def test_frequencies(crs):
    f = crs.rope_inv_freq(8, base=1e4, device="cpu")
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(crs.rope_inv_freq(8, factor=4.0, device="cpu"), f / 4, rtol=1e-14)
    b = crs.rope_inv_freq(8, factor=4.0, scaling="base", device="cpu")
    assert abs(float(b[0]) - 1.0) < 1e-15 and abs(float(b[-1]) * 4 / float(f[-1]) - 1) < 1e-12
    p = crs.rope_inv_freq(128, factor=8.0, scaling="parts", trained_len=4096, device="cpu")
    f = crs.rope_inv_freq(128, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(p[turns > 40], f[turns > 40])
    assert torch.allclose(p[turns < 0.5], f[turns < 0.5] / 8)
    assert (p <= f).all() and (p >= f / 8 * (1 - 1e-12)).all()
