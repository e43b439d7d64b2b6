"""Selection by accumulated weight, eviction, append and commit of the paged cache: whole
numbers and copied rows, so equality throughout (rotated rows: the rope tolerance)."""
import math

import pytest
import torch

import cache_ref as ref
from test_gpu_rope import limit

pytestmark = pytest.mark.gpu


def masses(g, *shape):
    m = torch.rand(shape, generator=g) ** 6
    m[torch.rand(shape, generator=g) < 0.1] = 0.0              # ties
    m[torch.rand(shape, generator=g) < 0.02] = -0.0
    return m


@pytest.mark.parametrize("cap", [1, 5, 100, 1024, 1025, 2048, 4000, 8192, 9000, 20000, 40000])
def test_select(crs, cuda_dev, cap):
    """Every register form and the memory form; lengths 0, 1, keep, keep + 1 and full."""
    g = torch.Generator().manual_seed(cap)
    for keep in sorted({1, max(1, cap // 3), cap}):
        lens = [0, 1, min(cap, keep), min(cap, keep + 1), cap, max(1, cap // 2)]
        n_kv = 2 if cap < 5000 else 1
        m = masses(g, len(lens), n_kv, cap)
        pos = torch.stack([torch.stack([torch.randperm(cap, generator=g) for _ in range(n_kv)])
                           for _ in lens]).to(torch.int32)
        sl = torch.tensor(lens, dtype=torch.int32)
        nxt = torch.full((len(lens),), cap, dtype=torch.int32)
        for kw in ({}, dict(pos=pos, next_pos=nxt, sink_end=min(2, keep // 2), window=min(7, keep // 2))):
            dkw = {k: (v.to(cuda_dev) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
            idx, cnt = crs.mass_select(m.to(cuda_dev), sl.to(cuda_dev), keep, **dkw)
            ei, ec = ref.select(m, sl, keep, **kw)
            assert torch.equal(cnt.cpu(), ec) and torch.equal(idx.cpu(), ei), (keep, kw.keys())
    assert crs.get_device_error() == 0


@pytest.mark.parametrize("cap", [900, 33000])
def test_select_special_values(crs, cuda_dev, cap):
    """Infinities, subnormals, equal keys throughout; a NaN is flagged and ranks last."""
    g = torch.Generator().manual_seed(5)
    m = torch.zeros(4, 1, cap)
    m[0] = 0.5
    m[1] = torch.tensor([math.inf, -math.inf, 1e-42, -1e-42, 0.0])[torch.randint(0, 5, (1, cap), generator=g)]
    m[2] = torch.randn(1, cap, generator=g)
    m[3] = -torch.rand(1, cap, generator=g)
    sl = torch.full((4,), cap - 3, dtype=torch.int32)
    for keep in (1, 130, cap - 4):
        idx, cnt = crs.mass_select(m.to(cuda_dev), sl.to(cuda_dev), keep)
        ei, ec = ref.select(m, sl, keep)
        assert torch.equal(idx.cpu(), ei) and torch.equal(cnt.cpu(), ec)
    assert crs.get_device_error() == 0
    m[2, 0, ::3] = float("nan")
    idx, _ = crs.mass_select(m.to(cuda_dev), sl.to(cuda_dev), cap - 100)
    assert torch.equal(idx.cpu(), ref.select(m, sl, cap - 100)[0])
    assert crs.get_device_error() == crs.DEVERR_NONFINITE


def test_select_lists_feed_sparse_attn(crs, cuda_dev):
    """The lists are what the gather attention reads (contiguous cache, one list per KV head)."""
    g = torch.Generator(device=cuda_dev).manual_seed(6)
    n_seq, n_kv, cap, D = 3, 2, 256, 128
    K = torch.randn(n_seq * cap, n_kv, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    V = torch.randn(n_seq * cap, n_kv, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    Q = torch.randn(n_seq, 8, D, generator=g, device=cuda_dev).to(torch.bfloat16)
    mass = torch.rand(n_seq, n_kv, cap, generator=g, device=cuda_dev)
    sl = torch.tensor([256, 100, 40], dtype=torch.int32, device=cuda_dev)
    idx, cnt = crs.mass_select(mass, sl, 64)
    base = torch.arange(n_seq, device=cuda_dev) * cap
    O, _ = crs.sparse_attn(Q, K, V, idx, kv_base=base)
    for s in range(n_seq):
        for h in range(8):
            j = idx[s, h // 4, : int(cnt[s])].long() + s * cap
            k, v = K[j, h // 4].double(), V[j, h // 4].double()
            e = torch.softmax(k @ Q[s, h].double() / math.sqrt(D), 0) @ v
            assert ((O[s, h].double() - e).abs() <= 2e-3 * e.abs().clamp(min=1.0)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,cap,keep", [(16, 64, 20), (24, 300, 200), (1, 33, 16), (64, 700, 513), (100, 100, 99)])
def test_evict(crs, cuda_dev, D, page, cap, keep):
    g = torch.Generator().manual_seed(page + keep)
    n_kv, lens = 3, [cap, 0, 1, keep, min(cap, keep + 1), cap // 2]
    n_seq, max_pages = len(lens), -(-cap // page)
    k = torch.randn(n_seq * max_pages, page, n_kv, D, generator=g).to(torch.bfloat16)
    v = torch.randn(n_seq * max_pages, page, n_kv, D, generator=g).to(torch.bfloat16)
    table = torch.randperm(n_seq * max_pages, generator=g).to(torch.int32).view(n_seq, max_pages)
    mass = masses(g, n_seq, n_kv, cap)
    pos = torch.randint(0, 9999, (n_seq, n_kv, cap), generator=g).to(torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32)
    idx, cnt = ref.select(mass, sl, keep)
    ek, ev, ep, em = ref.evict(k, v, table, pos, mass, idx, cnt)
    d = [t.to(cuda_dev) for t in (k, v, table, sl, sl, pos, mass)]
    d[4] = d[4].clone()
    cache = crs.KvCache(*d[:5], pos=d[5], mass=d[6])
    for _ in range(2):                                         # repeating it changes nothing
        cache.evict(idx.to(cuda_dev), cnt.to(cuda_dev))
        assert torch.equal(cache.k_pool.cpu(), ek) and torch.equal(cache.v_pool.cpu(), ev)
        assert torch.equal(cache.pos.cpu(), ep) and torch.equal(cache.mass.cpu(), em)
        assert torch.equal(cache.seq_len.cpu(), cnt) and torch.equal(cache.next_pos.cpu(), sl)
    assert crs.get_device_error() == 0


def test_evict_flags_bad_entries(crs, cuda_dev):
    k = torch.zeros(4, 8, 1, 64, dtype=torch.bfloat16, device=cuda_dev)
    table = torch.arange(4, dtype=torch.int32, device=cuda_dev).view(1, 4)
    sl = torch.tensor([32], dtype=torch.int32, device=cuda_dev)
    cache = crs.KvCache(k, k.clone(), table, sl, sl.clone())
    idx = torch.tensor([[[0, 5, 40, 10 ** 9]]], dtype=torch.int32, device=cuda_dev)
    cache.evict(idx, torch.tensor([99], dtype=torch.int32, device=cuda_dev))      # count cut to keep
    torch.cuda.synchronize()
    assert crs.get_device_error() == crs.DEVERR_INDEX
    assert int(cache.seq_len[0]) == 4


@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, True), (128, 48, False), (64, 0, False)])
@pytest.mark.parametrize("n_tok", [1, 5, 130])
def test_append_and_commit(crs, cuda_dev, D, rot, inter, n_tok):
    g = torch.Generator().manual_seed(rot + n_tok)
    n_seq, n_kv, n_q, page, cap = 5, 2, 6, 12, 160
    max_pages = -(-cap // page)
    k0 = torch.randn(n_seq * max_pages, page, n_kv, D, generator=g).to(torch.bfloat16)
    v0 = torch.randn(n_seq * max_pages, page, n_kv, D, generator=g).to(torch.bfloat16)
    table = torch.randperm(n_seq * max_pages, generator=g).to(torch.int32).view(n_seq, max_pages)
    sl = torch.tensor([0, 11, 12, cap - 1, 25], dtype=torch.int32)
    nxt = torch.tensor([1000, 0, 77, 10 ** 6, 25], dtype=torch.int32)
    n_new = torch.tensor([n_tok, 0, n_tok, n_tok, max(0, n_tok - 1)], dtype=torch.int32)
    qkv = torch.randn(n_seq, n_tok, n_q + 2 * n_kv, D, generator=g).to(torch.bfloat16)
    q, k, v = qkv[:, :, :n_q], qkv[:, :, n_q:n_q + n_kv], qkv[:, :, n_q + n_kv:]
    f = crs.rope_inv_freq(rot, base=1e4, device="cpu") if rot else None
    pos = torch.full((n_seq, n_kv, cap), -7, dtype=torch.int32)
    mass = torch.ones(n_seq, n_kv, cap)
    dev = lambda t: t.to(cuda_dev)  # noqa: E731
    cache = crs.KvCache(dev(k0), dev(v0), dev(table), dev(sl), dev(nxt), pos=dev(pos), mass=dev(mass))
    d = dev(qkv)                                               # strided slices of one projection
    q_out = cache.append(d[:, :, n_q:n_q + n_kv], d[:, :, n_q + n_kv:], q=d[:, :, :n_q],
                         inv_freq=None if f is None else dev(f), n_new=dev(n_new), interleaved=inter)
    torch.cuda.synchronize()
    used = ref.n_used(n_new, n_tok, sl, cap)
    over = any(u < min(int(n), n_tok) for u, n in zip(used, n_new))
    assert crs.get_device_error() == (crs.DEVERR_CAPACITY if over else 0)
    ek, ev, ep, em = k0.clone(), v0.clone(), pos.clone(), mass.clone()
    eq = torch.zeros(n_seq, n_tok, n_q, D, dtype=torch.float64)
    tk = torch.zeros(ek.shape, dtype=torch.float64)
    tq = torch.zeros(eq.shape, dtype=torch.float64)
    ek = ek.double()
    for s in range(n_seq):
        for i in range(used[s]):
            p = nxt[s] + i
            j = int(sl[s]) + i
            at = (int(table[s, j // page]), j % page)
            for src, dst, t, w in ((k[s, i], ek, tk, at), (q[s, i], eq, tq, (s, i))):
                if f is None:
                    dst[w] = src.double()
                else:
                    dst[w] = ref.rope(src[None], p[None], f, 0, inter)[0]
                    t[w] = limit(src, dst[w], f, 0, inter, 1.0)
            ev[at] = v[s, i]
            ep[s, :, j] = p
            em[s, :, j] = 0.0
    assert ((cache.k_pool.double().cpu() - ek).abs() <= tk).all()
    assert ((q_out.double().cpu() - eq).abs() <= tq).all()
    assert torch.equal(cache.v_pool.cpu(), ev) and torch.equal(cache.pos.cpu(), ep) and torch.equal(cache.mass.cpu(), em)
    assert torch.equal(cache.seq_len.cpu(), sl) and torch.equal(cache.next_pos.cpu(), nxt)
    acc = torch.tensor([n_tok, 1, -4, n_tok, 0], dtype=torch.int32)
    cache.commit(dev(acc), n_tok=n_tok)
    eff = torch.tensor(ref.n_used(acc, n_tok, sl, cap), dtype=torch.int32)
    assert torch.equal(cache.seq_len.cpu(), sl + eff) and torch.equal(cache.next_pos.cpu(), nxt + eff)
    before = cache.seq_len.cpu()
    cache.commit(1)
    assert torch.equal(cache.seq_len.cpu(), (before + 1).clamp(max=cap))


def test_a_generation_with_eviction(crs, cuda_dev):
    """The operators as a loop uses them, against the 64-bit forms of all of them: a shared
    prefix, a ragged prompt chunk, then steps; every few steps the heads shrink to a budget.
    The reference follows the library's own lists (a near tie may order differently in fp32)."""
    g = torch.Generator().manual_seed(11)
    n_seq, n_kv, n_q, D, plen, cap, keep, page = 3, 2, 4, 64, 90, 48, 24, 8
    r = lambda *sh: torch.randn(sh, generator=g).to(torch.bfloat16)  # noqa: E731
    pk, pv = r(plen, n_kv, D), r(plen, n_kv, D)
    cache = crs.KvCache.empty(n_seq, n_kv, cap, D=D, page_size=page, first_pos=plen, device=cuda_dev)
    f = crs.rope_inv_freq(D, base=1e4)
    dpk, dpv = pk.to(cuda_dev), pv.to(cuda_dev)
    mass_bound = torch.zeros(n_seq, n_kv, cap, dtype=torch.float64)
    for step in range(30):
        n_tok = 10 if step == 0 else 1
        n_new = torch.tensor([10, 3, 7], dtype=torch.int32, device=cuda_dev) if step == 0 else None
        q, k, v = r(n_seq, n_tok, n_q, D), r(n_seq, n_tok, n_kv, D), r(n_seq, n_tok, n_kv, D)
        qr = cache.append(k.to(cuda_dev), v.to(cuda_dev), q=q.to(cuda_dev), inv_freq=f, n_new=n_new)
        before = cache.mass.cpu()
        O, lse = cache.attend(qr, dpk, dpv, n_new=n_new, mass_out=cache.mass)
        eO, el, em, A = ref.attend(qr.cpu(), cache.k_pool.cpu(), cache.v_pool.cpu(), cache.block_table.cpu(),
                                   cache.seq_len.cpu(), cap, None if n_new is None else n_new.cpu(), pk, pv,
                                   mass=before)
        assert ((O.double().cpu() - eO).abs() <= A * 2.0 ** -13 + 1e-30).all()
        assert ((cache.mass.double().cpu() - em).abs() <= (em - before.double()).abs() * 2.0 ** -14 +
                em.abs() * 2.0 ** -21).all()
        cache.commit(n_tok if n_new is None else n_new, n_tok=n_tok)
        if int(cache.seq_len.max()) >= 40:
            idx, cnt = cache.select(keep, window=4)
            ei, ec = ref.select(cache.mass.cpu(), cache.seq_len.cpu(), keep, cache.pos.cpu(), cache.next_pos.cpu(),
                                0, 4)
            assert torch.equal(idx.cpu(), ei) and torch.equal(cnt.cpu(), ec)
            ek, ev, ep, em = ref.evict(cache.k_pool.cpu(), cache.v_pool.cpu(), cache.block_table.cpu(),
                                       cache.pos.cpu(), cache.mass.cpu(), ei, ec)
            cache.evict(idx, cnt)
            assert torch.equal(cache.k_pool.cpu(), ek) and torch.equal(cache.v_pool.cpu(), ev)
            assert torch.equal(cache.pos.cpu(), ep) and torch.equal(cache.mass.cpu(), em)
    assert crs.get_device_error() == 0
    assert int(cache.next_pos[0]) == plen + 10 + 29 and int(cache.seq_len[0]) < 40


def test_replaced_tensors_are_used(crs, cuda_dev):
    """Every call after `cache.x = new` reads and writes the new tensor, and only it."""
    g = torch.Generator().manual_seed(31)
    n_seq, n_kv, D, cap = 3, 2, 64, 32
    r = lambda *sh: torch.randn(sh, generator=g).to(torch.bfloat16).to(cuda_dev)  # noqa: E731
    old = crs.KvCache.empty(n_seq, n_kv, cap, D=D, page_size=8, device=cuda_dev)
    new = crs.KvCache.empty(n_seq, n_kv, cap, D=D, page_size=8, first_pos=5, device=cuda_dev)
    new.block_table.copy_(new.block_table.flip(0))
    names = ("k_pool", "v_pool", "block_table", "pos", "mass", "seq_len", "next_pos")
    kept = {n: getattr(old, n).clone() for n in names}
    first = {n: getattr(old, n) for n in names}
    want = crs.KvCache(*(getattr(new, n).clone() for n in ("k_pool", "v_pool", "block_table", "seq_len", "next_pos")),
                       pos=new.pos.clone(), mass=new.mass.clone())
    for n in names:
        setattr(old, n, getattr(new, n))
    f = crs.rope_inv_freq(D)
    for _ in range(12):
        q, k, v = r(n_seq, 2, 4, D), r(n_seq, 2, n_kv, D), r(n_seq, 2, n_kv, D)
        outs = []
        for c in (old, want):
            qr = c.append(k, v, q=q, inv_freq=f)
            outs.append((qr,) + c.attend(qr, mass_out=c.mass))
            c.commit(2)
        assert all(torch.equal(a, b) for a, b in zip(*outs))
    for c in (old, want):
        c.evict(*c.select(10, window=2))
    for n in names:
        assert torch.equal(getattr(old, n), getattr(want, n))
        assert torch.equal(first[n], kept[n])                  # the replaced ones are left alone
    assert crs.get_device_error() == 0


def test_many_heads(crs, cuda_dev):
    """4096 sequences of 17 heads, four slots each, two kept: more (sequence, head) pairs than a
    grid's second dimension holds."""
    g = torch.Generator(device=cuda_dev).manual_seed(41)
    n_seq, n_kv, D = 4096, 17, 64
    cache = crs.KvCache.empty(n_seq, n_kv, 4, D=D, page_size=4, device=cuda_dev)
    for t in (cache.k_pool, cache.v_pool):
        t.copy_(torch.randint(-99, 99, t.shape, generator=g, device=cuda_dev))
    cache.mass.copy_(torch.rand(cache.mass.shape, generator=g, device=cuda_dev))
    cache.pos.copy_(torch.randint(0, 99, cache.pos.shape, generator=g, device=cuda_dev))
    cache.seq_len.fill_(4)
    idx, count = crs.mass_select(cache.mass, cache.seq_len, 2)       # by weight alone
    best = cache.mass.sort(dim=-1, descending=True, stable=True).indices[..., :2].sort(dim=-1).values
    assert torch.equal(idx.long(), best) and (count == 2).all()
    # what slots 0 and 1 hold afterwards: themselves, or the r-th kept slot past them
    a, b = best.unbind(-1)
    first = torch.where(a == 0, a, torch.where(a == 1, b, a))
    second = torch.where(a == 1, a, b)
    src = torch.stack([first, second, torch.full_like(a, 2), torch.full_like(a, 3)], -1)
    at = src.transpose(1, 2)[..., None].expand(-1, -1, -1, D)
    want = [t.view(n_seq, 4, n_kv, D).gather(1, at) for t in (cache.k_pool, cache.v_pool)]
    want += [t.gather(2, src) for t in (cache.pos, cache.mass)]
    cache.evict(idx, count)
    got = [t.view(n_seq, 4, n_kv, D) for t in (cache.k_pool, cache.v_pool)] + [cache.pos, cache.mass]
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and (cache.seq_len == 2).all()
    assert crs.get_device_error() == 0
