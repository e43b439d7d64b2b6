"""Frequencies stretched by parts, against the rule pair by pair (CPU only)."""
import math

import pytest
import torch


@pytest.mark.parametrize("rot_dim", [32, 64, 128])
@pytest.mark.parametrize("base", [1e4, 5e5])
@pytest.mark.parametrize("trained_len", [24, 128, 4096, 131072, 2 ** 20])
@pytest.mark.parametrize("factor", [4.0, 32.0])
def test_parts_follow_the_turns(crs, rot_dim, base, trained_len, factor):
    """Pairs of more than beta_fast turns are left, of fewer than beta_slow divided, and every
    pair between is between; the slowest pair may make many turns, the fastest few."""
    f = crs.rope_inv_freq(rot_dim, base=base, device="cpu")
    p = crs.rope_inv_freq(rot_dim, base=base, factor=factor, scaling="parts", trained_len=trained_len, device="cpu")
    turns = f * trained_len / (2 * math.pi)
    fast, slow = turns >= 32.0, turns <= 1.0
    assert torch.equal(p[fast], f[fast])
    assert torch.allclose(p[slow], f[slow] / factor, rtol=1e-14)
    mid = ~fast & ~slow
    share = (f - p) / (f - f / factor)           # 0: left, 1: divided
    assert (share[1:] >= share[:-1] - 1e-12).all()
    # the blend is linear in the pair's index between the pairs of 32 turns and of 1, whose
    # indices are rounded outwards: both ends off by less than one pair
    pair = lambda t: rot_dim * math.log(trained_len / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
    j = torch.arange(rot_dim // 2, dtype=torch.float64)
    assert ((share - (j - lo) / (hi - lo))[mid].abs() <= 1e-9).all()
    assert ((share[mid] > 0) & (share[mid] < 1)).all()


def test_parts_of_a_long_trained_length(crs):
    """2.4 turns of the slowest pair over 131072 positions: blended, not divided."""
    f = crs.rope_inv_freq(128, base=1e4, device="cpu")
    p = crs.rope_inv_freq(128, base=1e4, factor=8.0, scaling="parts", trained_len=131072, device="cpu")
    assert float(f[-1]) * 131072 / (2 * math.pi) > 2.4
    assert float(p[-1]) > 1.5 * float(f[-1]) / 8.0


def test_parts_with_one_border(crs):
    """beta_fast = beta_slow: a step."""
    f = crs.rope_inv_freq(128, device="cpu")
    p = crs.rope_inv_freq(128, factor=2.0, scaling="parts", trained_len=4096, beta_fast=8.0, beta_slow=8.0, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(p[turns > 8.0], f[turns > 8.0]) and torch.equal(p[turns < 8.0], f[turns < 8.0] / 2)
