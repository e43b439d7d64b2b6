"""The 24 bits that an f32 output of the cache attention keeps: of its weights (three bf16 parts)
and of its sums (short chains of tensor-core additions, which truncate)."""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu


def small(g, *shape):
    """Whole numbers of [-8, 8]."""
    return torch.randint(-8, 9, shape, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where,n_seq", [("prefix", 40), ("prefix", 4), ("slots", 6)])
def test_two_keys_share_a_row(crs, cuda_dev, D, where, n_seq):
    """Two keys count, the others are 56 or more below them (less than 2^-70 together).  Their dot
    products are whole numbers (exact), logits z2 in log2 units up to Z.  A weight is off by
    ln 2 2^-24 6 Z at most (the scale's rounding, the product's, the difference's, for both keys)
    and ex2.approx's 2^-22; the denominator doubles that; the parts of the weights leave 2^-26
    each, their three additions truncate 2^-23 each, and the merge rounds three times: 2^-21.
    Without the third part a weight would be off by up to 2^-17 of its binade.
    160 and 16 query rows per KV head: the tensor-core prefix and the plain one."""
    g = torch.Generator().manual_seed(51)
    n_kv, G, n, scale = 2, 4, 300, 2.0 ** -10
    q = small(g, n_seq, 1, n_kv * G, D)
    q[..., 0] = 240.0
    far = torch.zeros(n, n_kv, D, dtype=torch.bfloat16)
    far[..., 0] = -240.0
    keys = far.clone()
    for j in (5, 201):
        keys[j] = small(g, n_kv, D)
        keys[j, :, 0] = 0.0
    values = torch.randn(n, n_kv, D, generator=g).to(torch.bfloat16)
    cache = crs.KvCache.empty(n_seq, n_kv, n, D=D, page_size=16, device=cuda_dev)
    pk = pv = None
    if where == "prefix":
        pk, pv = keys, values
        own_k, own_v, lens = far[:3], values[:3], 2
    else:
        own_k, own_v, lens = keys, values, n - 1
    rows = torch.zeros(n_seq, cache.block_table.shape[1] * 16, n_kv, D, dtype=torch.bfloat16)
    for pool, src in ((cache.k_pool, own_k), (cache.v_pool, own_v)):
        rows.zero_()
        rows[:, :len(src)] = src
        pool.copy_(rows.view(pool.shape))
    cache.seq_len.fill_(lens)
    dev = lambda t: None if t is None else t.to(cuda_dev)  # noqa: E731
    O, _ = cache.attend(q.to(cuda_dev), dev(pk), dev(pv), scale=scale)
    eO, _, _, A = ref.attend(q, cache.k_pool.cpu(), cache.v_pool.cpu(), cache.block_table.cpu(), cache.seq_len.cpu(),
                             n, pk=pk, pv=pv, scale=scale)
    near = keys[[5, 201]].double()
    z2 = torch.einsum("sihgd,jhd->sihgj", q.view(n_seq, 1, n_kv, G, D).double(), near) * scale * math.log2(math.e)
    tol = 2.0 * (math.log(2.0) * 2.0 ** -24 * 6.0 * float(z2.abs().max()) + 2.0 ** -22) + 2.0 ** -21
    assert tol < 2.0 ** -18
    assert ((O.double().cpu() - eO).abs() <= A * tol + eO.abs() * 2.0 ** -24).all()
    assert crs.get_device_error() == 0


def test_a_long_prefix_adds_up(crs, cuda_dev):
    """Every key has the same value v, so the output is v whatever the weights are, but for the sums:
    a chain of at most 640 keys adds 3 parts per 16 of them and truncates 2^-23 each time
    (120 2^-23), the merge of 50 pieces rounds 100 times by 2^-24, and the denominator's chains of
    at most 28 and then 50 additions likewise: 120 + (100 + 78 + 10) / 2 steps of 2^-23 in all.  One
    chain over half of the 32000 keys would lose some 900 steps (3000 truncations of an average 0.3)."""
    n_seq, n_kv, n_q, D, n = 320, 8, 64, 128, 32000
    g = torch.Generator(device=cuda_dev).manual_seed(52)
    q = torch.randn(n_seq, 1, n_q, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    pk = torch.randn(n, n_kv, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    v = (1.0 + torch.rand(n_kv, D, generator=g, device=cuda_dev)).to(torch.bfloat16)
    cache = crs.KvCache.empty(n_seq, n_kv, 16, D=D, page_size=16, device=cuda_dev)
    cache.v_pool.copy_(v.expand(cache.v_pool.shape))
    O, _ = cache.attend(q, pk, v.expand(n, n_kv, D).contiguous())
    e = v.double().repeat_interleave(n_q // n_kv, 0)
    err = (O.double() / e - 1.0).abs().max()
    assert float(err) <= (120 + (100 + 78 + 10) / 2) * 2.0 ** -23
    assert crs.get_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_long_slots_add_up(crs, cuda_dev, D):
    """The same for 20000 own slots (all sequences on the same pages): a tile's 16 keys of a warp
    truncate three times (3 2^-23, to one side), the tiles are added up with rounding, to
    either side, so that the mean over 512 x 4 rows is off by less than another 2^-23.  One chain
    of 313 tiles would lose some 280 2^-23 (940 truncations of an average 0.3)."""
    n_seq, n_kv, n_q, n, page = 64, 8, 32, 20000, 64
    g = torch.Generator(device=cuda_dev).manual_seed(53)
    pages = -(-n // page)
    k = torch.randn(pages, page, n_kv, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    v = (1.0 + torch.rand(n_kv, D, generator=g, device=cuda_dev)).to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32, device=cuda_dev).repeat(n_seq, 1)
    sl = torch.full((n_seq,), n - 1, dtype=torch.int32, device=cuda_dev)
    cache = crs.KvCache(k, v.expand(pages, page, n_kv, D).contiguous(), table, sl, sl.clone())
    q = torch.randn(n_seq, 1, n_q, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    O, _ = cache.attend(q)
    e = v.double().repeat_interleave(n_q // n_kv, 0)
    err = O.double() / e - 1.0
    assert abs(float(err.mean())) <= 4 * 2.0 ** -23
    assert float(err.abs().max()) <= 2.0 ** -15
    assert crs.get_device_error() == 0
