"""Decode attention over a shared prefix and the cached slots, against the 64-bit form.

Tolerances.  With exact weights p_j (sum 1) and output O = sum p_j v_j, A = sum p_j |v_j|:
 * a logit z (in log2 units, |z| <= Z) carries an fp32 error of at most
   D 2^-24 sum|q_i k_i| scale log2(e) + 2 |z| 2^-24 (products exact, D additions, the scale) and
   the subtraction of the maximum another |z - m| 2^-24; for normal inputs at scale 1/sqrt(D) this
   is below 2^-16 relative in p, with ex2.approx's 2^-22.  The same error of the denominator
   doubles it: 2^-15 A.
 * sums of the weights and of p v: chains of at most 2^7 tensor-core steps per piece with at most
   one fp32 step (2^-23, truncated) each, and a few joins: 2^-15 A.
 * weights rounded to bf16 (half a step: 2^-8 relative before normalisation): 2^-8 A; split into
   three bf16 parts: the last residual's half step, below the 2^-17 A allowed here.
 * the output's own half step: 2^-8 |O| in bf16, 2^-24 |O| in f32.
So |O' - O| <= A (2^-14 + 2^-17) for f32, A (2^-14 + 2^-8) + 2^-8 |O| for bf16; lse is off by
2^-15 + |lse| 2^-22, an accumulated weight by 2^-14 of the sum of its contributions and 2^-23 of
the result per addition.
"""
import math

import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu

TOL_F32 = 2.0 ** -14 + 2.0 ** -17


def make(dev, n_seq, n_tok, n_q, n_kv, D, page, lens, prefix, seed, ragged=False, cap=None, poison=True,
         spread=1.0):
    """A cache with shuffled pages whose unused rows hold NaN and infinities."""
    g = torch.Generator().manual_seed(seed)
    cap = max(lens) + n_tok if cap is None else cap
    max_pages = -(-cap // page)
    n_pages = n_seq * max_pages + 3
    r = lambda *sh: torch.randn(sh, generator=g).to(torch.bfloat16)  # noqa: E731
    k, v = r(n_pages, page, n_kv, D) * spread, r(n_pages, page, n_kv, D)
    table = torch.randperm(n_pages, generator=g)[: n_seq * max_pages].to(torch.int32).view(n_seq, max_pages)
    n_new = torch.randint(0, n_tok + 1, (n_seq,), generator=g).to(torch.int32) if ragged else None
    used = ref.n_used(n_new, n_tok, lens, cap)
    if poison:
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        for s in range(n_seq):
            for j in range(lens[s] + used[s]):
                live[int(table[s, j // page]), j % page] = True
        k[~live] = float("nan")
        v[~live] = float("inf")
    q = r(n_seq, n_tok, n_q, D) * spread
    pk, pv = (r(prefix, n_kv, D) * spread, r(prefix, n_kv, D)) if prefix else (None, None)
    mass = torch.rand((n_seq, n_kv, cap), generator=g)
    pos = torch.arange(cap, dtype=torch.int32).repeat(n_seq, n_kv, 1)
    sl = torch.tensor(lens, dtype=torch.int32)
    return dict(k=k, v=v, table=table, n_new=n_new, q=q, pk=pk, pv=pv, mass=mass, pos=pos, seq_len=sl, cap=cap,
                used=used)


def on(dev, c, crs):
    d = {n: (t.to(dev) if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    cache = crs.KvCache(d["k"], d["v"], d["table"], d["seq_len"], d["seq_len"].clone(), pos=d["pos"], mass=d["mass"])
    return d, cache


def check(crs, dev, c, out_dtype, with_mass=True, decay=1.0, scale=None):
    d, cache = on(dev, c, crs)
    mo = d["mass"].clone() if with_mass else None
    O, lse = cache.attend(d["q"], d["pk"], d["pv"], n_new=d["n_new"], out_dtype=out_dtype, mass_out=mo, decay=decay,
                          scale=scale)
    torch.cuda.synchronize()
    assert crs.get_device_error() == 0
    eO, el, em, A = ref.attend(c["q"], c["k"], c["v"], c["table"], c["seq_len"], c["cap"], c["n_new"], c["pk"],
                               c["pv"], scale=scale, mass=c["mass"], decay=decay)
    o = O.double().cpu()
    tol = A * TOL_F32 + eO.abs() * 2.0 ** -24 if out_dtype == torch.float32 else \
        A * (2.0 ** -14 + 2.0 ** -8) + eO.abs() * 2.0 ** -8
    bad = ((o - eO).abs() > tol) | ~torch.isfinite(o)
    assert not bad.any(), (int(bad.sum()), float((o - eO).abs().max()))
    l = lse.double().cpu()
    assert torch.equal(torch.isfinite(l), torch.isfinite(el))
    f = torch.isfinite(el)
    assert ((l[f] - el[f]).abs() <= 2.0 ** -15 + el[f].abs() * 2.0 ** -22).all()
    assert torch.equal(l[~f], el[~f])
    if with_mass:
        got = mo.double().cpu()
        tol = (em - decay * c["mass"].double()).abs() * 2.0 ** -14 + em.abs() * 2.0 ** -21
        for s in range(len(c["used"])):
            t = int(c["seq_len"][s]) + c["used"][s]
            assert ((got - em).abs() <= tol)[s, :, :t].all()
            assert torch.equal(mo[s, :, t:].cpu(), c["mass"][s, :, t:])     # other slots untouched
    return d, cache, O, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_q,n_kv", [(4, 4), (6, 2), (16, 1)])
def test_own_slots_only(crs, cuda_dev, D, out_dtype, n_q, n_kv):
    """No prefix; lengths of zero, one, and around the tile and page borders."""
    c = make(cuda_dev, 6, 1, n_q, n_kv, D, 24, [0, 1, 62, 63, 64, 200], 0, 1)
    check(crs, cuda_dev, c, out_dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 300])
def test_prefix_and_slots(crs, cuda_dev, D, out_dtype, prefix):
    c = make(cuda_dev, 5, 1, 8, 2, D, 16, [0, 5, 64, 65, 129], prefix, 2)
    check(crs, cuda_dev, c, out_dtype)


@pytest.mark.parametrize("n_tok,n_q,n_kv", [(2, 4, 2), (5, 12, 4), (3, 40, 2), (7, 21, 3)])
def test_several_new_tokens(crs, cuda_dev, n_tok, n_q, n_kv):
    """Causal among the new tokens; more query rows than one tile; some sequences without any."""
    for ragged in (False, True):
        c = make(cuda_dev, 4, n_tok, n_q, n_kv, 128, 7, [0, 9, 63, 100], 77, 3, ragged=ragged)
        check(crs, cuda_dev, c, torch.float32, decay=0.5)


@pytest.mark.parametrize("n_seq,prefix", [(40, 700), (90, 130), (33, 1)])
def test_many_sequences_share_the_prefix(crs, cuda_dev, n_seq, prefix):
    """The prefix's query tile holds the whole batch, past 128 rows too."""
    lens = [(7 * s) % 50 for s in range(n_seq)]
    c = make(cuda_dev, n_seq, 1, 8, 2, 128, 32, lens, prefix, 4)
    check(crs, cuda_dev, c, torch.bfloat16)
    check(crs, cuda_dev, c, torch.float32, with_mass=False)


def test_rows_that_see_nothing(crs, cuda_dev):
    """No new token and no prefix: zeros, -inf, and the mass as it was."""
    c = make(cuda_dev, 3, 2, 4, 2, 64, 16, [0, 5, 0], 0, 5)
    c["n_new"] = torch.tensor([0, -3, 9], dtype=torch.int32)          # cut to 0, 0, 2
    c["used"] = ref.n_used(c["n_new"], 2, [0, 5, 0], c["cap"])
    c["k"], c["v"] = torch.nan_to_num(c["k"]), torch.nan_to_num(c["v"], posinf=0.0)
    d, cache, O, lse = check(crs, cuda_dev, c, torch.float32)
    assert (O[:2] == 0).all() and torch.isinf(lse[:2]).all()


def test_wide_logits(crs, cuda_dev):
    """Logits of some hundreds: the running maximum moves, far weights vanish."""
    c = make(cuda_dev, 4, 1, 8, 2, 128, 16, [3, 70, 150, 500], 400, 6, spread=6.0)
    d, cache = on(cuda_dev, c, crs)
    O, lse = cache.attend(d["q"], d["pk"], d["pv"])
    eO, el, _, A = ref.attend(c["q"], c["k"], c["v"], c["table"], c["seq_len"], c["cap"], None, c["pk"], c["pv"])
    # |z| up to about 6 * 36 * sqrt(128) / sqrt(128) * 6 = 2^11 log2 units: 2^-24 2^11 D^(1/2) < 2^-9 relative in p
    assert ((O.double().cpu() - eO).abs() <= A * 2.0 ** -8 + 1e-30).all()
    assert ((lse.double().cpu() - el).abs() <= el.abs() * 2.0 ** -18 + 2.0 ** -15).all()


def test_full_cache_drops_the_last_tokens(crs, cuda_dev):
    c = make(cuda_dev, 2, 3, 4, 2, 64, 8, [14, 3], 20, 7, cap=16)
    check(crs, cuda_dev, c, torch.float32)


def test_bad_page_is_flagged_and_skipped(crs, cuda_dev):
    """A block table entry outside the pool: its slots are skipped, the error word says so."""
    c = make(cuda_dev, 1, 1, 2, 2, 64, 8, [20], 0, 8, poison=False)
    c["table"][0, 1] = 10 ** 6
    d, cache = on(cuda_dev, c, crs)
    O, lse = cache.attend(d["q"])
    torch.cuda.synchronize()
    assert crs.get_device_error() == crs.DEVERR_INDEX
    K = torch.stack([c["k"][int(c["table"][0, j // 8]), j % 8] for j in range(21) if j // 8 != 1]).double()
    z = torch.einsum("jhd,hd->hj", K, c["q"][0, 0].double()) / 8.0
    assert ((lse[0, 0].double().cpu() - torch.logsumexp(z, 1)).abs() <= 2.0 ** -14).all()


def test_streams_graphs_and_repeats(crs, cuda_dev):
    """The same bits again, on another stream, and from a captured graph after the lengths moved."""
    c = make(cuda_dev, 7, 1, 8, 4, 128, 16, [0, 1, 30, 64, 77, 128, 300], 500, 9, poison=False, cap=320)
    d, cache = on(cuda_dev, c, crs)
    mo = d["mass"].clone()
    O, lse = cache.attend(d["q"], d["pk"], d["pv"], mass_out=mo)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mo2 = d["mass"].clone()
    s.wait_stream(torch.cuda.current_stream())
    O2, lse2 = cache.attend(d["q"], d["pk"], d["pv"], mass_out=mo2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(mo, mo2)
    g = torch.cuda.CUDAGraph()
    out, ls, m3 = torch.empty_like(O), torch.empty_like(lse), d["mass"].clone()
    ws = torch.empty(cache.attend_workspace_size(8, 1, 500, with_mass=True), dtype=torch.uint8, device=cuda_dev)
    with torch.cuda.graph(g):
        cache.attend(d["q"], d["pk"], d["pv"], out=out, lse=ls, mass_out=m3, workspace=ws)
    d["seq_len"].copy_(torch.tensor([5, 0, 64, 63, 299, 1, 10], dtype=torch.int32))
    g.replay()
    mo4 = d["mass"].clone()
    O4, lse4 = cache.attend(d["q"], d["pk"], d["pv"], mass_out=mo4)
    torch.cuda.synchronize()
    assert torch.equal(out, O4) and torch.equal(ls, lse4)
    for s_ in range(7):
        t = int(d["seq_len"][s_]) + 1
        assert torch.equal(m3[s_, :, :t], mo4[s_, :, :t])


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_seq,prefix", [(9, 127), (9, 128), (9, 129), (9, 1500), (70, 257), (130, 640)])
def test_tensor_core_prefix(crs, cuda_dev, out_dtype, D, n_seq, prefix):
    """36, 280 and 520 rows per KV head: one stream pair, several row tiles, one, few and many
    key tiles, tails of one key."""
    lens = [(5 * s) % 20 for s in range(n_seq)]
    c = make(cuda_dev, n_seq, 1, 8, 2, D, 8, lens, prefix, 12)
    check(crs, cuda_dev, c, out_dtype, with_mass=False)


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1.0])
def test_tensor_core_prefix_scales(crs, cuda_dev, scale):
    """A negative and a zero scale; and logits wide enough to move the running shift."""
    c = make(cuda_dev, 20, 1, 8, 2, 128, 8, [3] * 20, 900, 13, spread=1.5 if scale == 1.0 else 1.0)
    d, cache = on(cuda_dev, c, crs)
    O, lse = cache.attend(d["q"], d["pk"], d["pv"], scale=scale)
    eO, el, _, A = ref.attend(c["q"], c["k"], c["v"], c["table"], c["seq_len"], c["cap"], None, c["pk"], c["pv"],
                              scale=scale)
    # |z| <= 2^8 log2 units here (1.5^2 * 128^(1/2) * 6 sigma * 1.44): 2^-24 2^8 a few times over
    assert ((O.double().cpu() - eO).abs() <= A * 2.0 ** -13 + 1e-30).all()
    assert ((lse.double().cpu() - el).abs() <= el.abs() * 2.0 ** -20 + 2.0 ** -14).all()


def test_forced_wait_timeout_of_the_prefix_pass(crs, cuda_dev):
    """The bounded waits' failure path: flagged, recorded, drained; the next call is right."""
    c = make(cuda_dev, 9, 1, 8, 2, 128, 8, [4] * 9, 600, 14)
    d, cache = on(cuda_dev, c, crs)
    crs.get_device_error()
    crs.get_device_diag()
    try:
        crs.debug_force_wait_timeout(True)
        cache.attend(d["q"], d["pk"], d["pv"])
        flags, diag = crs.get_device_error(), crs.get_device_diag()
    finally:
        crs.debug_force_wait_timeout(False)
    assert flags & crs.DEVERR_TIMEOUT
    assert diag[0] > 0 and diag[1] == 1
    check(crs, cuda_dev, c, torch.float32)


@pytest.mark.parametrize("n_seq,n_tok", [(129, 1), (300, 1), (260, 2)])
def test_more_sequences_than_a_block_keeps(crs, cuda_dev, n_seq, n_tok):
    """Past 128 sequences the lengths are scanned in pieces; many of them empty."""
    lens = [(s * 37) % 91 if s % 3 else 0 for s in range(n_seq)]
    c = make(cuda_dev, n_seq, n_tok, 2, 1, 64, 16, lens, 0, 15, ragged=n_tok > 1)
    check(crs, cuda_dev, c, torch.float32)


def test_two_streams_and_a_graph_at_once(crs, cuda_dev):
    """The chained kernels of two calls on two streams, and of a captured graph beside them,
    keep apart: every run has the bits of a lone one."""
    cs = [make(cuda_dev, 24, 1, 8, 2, 128, 16, [(11 * s + k) % 150 for s in range(24)], 700 + k, 16 + k,
               poison=False) for k in range(3)]
    runs = [on(cuda_dev, c, crs) for c in cs]
    alone = []
    for d, cache in runs:
        m = d["mass"].clone()
        alone.append(cache.attend(d["q"], d["pk"], d["pv"], out_dtype=torch.bfloat16, mass_out=m) + (m,))
    torch.cuda.synchronize()
    d, cache = runs[2]
    gm = d["mass"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = cache.attend(d["q"], d["pk"], d["pv"], out_dtype=torch.bfloat16, mass_out=gm)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        out = []
        for (d, cache), s in zip(runs[:2], streams):
            with torch.cuda.stream(s):
                m = d["mass"].clone()
                out.append(cache.attend(d["q"], d["pk"], d["pv"], out_dtype=torch.bfloat16, mass_out=m) + (m,))
        with torch.cuda.stream(streams[2]):
            gm.copy_(runs[2][0]["mass"])
            graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out + [(go, gl, gm)], alone):
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    assert crs.get_device_error() == 0


def large_logits(c, n_seq, D, sign, own):
    """Whole-numbered queries and keys, whose products are exact in fp32: dot products around
    +-D 48^2, a few steps of 48 apart, so that several keys of a row count.  The own slots lie
    `own` steps of about 48 above (below) the prefix."""
    g = torch.Generator().manual_seed(21)
    bump = lambda t: (torch.rand(t.shape, generator=g) < 1 / 64).float() * torch.where(  # noqa: E731
        torch.rand(t.shape, generator=g) < 0.5, 1.0, -1.0)
    c["q"] = torch.randint(40, 57, c["q"].shape, generator=g).to(torch.bfloat16)
    c["pk"] = (sign * 48 + bump(c["pk"])).to(torch.bfloat16)
    k = sign * 48 + bump(c["k"])
    k[..., :abs(own)] += 1.0 if own > 0 else -1.0
    c["k"] = k.to(torch.bfloat16)
    return c


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [0.125, 1.0])
@pytest.mark.parametrize("n_seq", [20, 70])
def test_tensor_core_prefix_large_logits(crs, cuda_dev, out_dtype, D, scale, n_seq):
    """Logits of 1.8e4 to 3e5 (natural), of both signs and rising from one to the other, with the
    own slots above, at and below the prefix: 80 and 280 query rows per KV head.

    The products are whole numbers below 2^24, exact in fp32.  The scaled logit of a slot is
    rounded once, half a step of |z|: 2^-24 |z| relative in its weight, as much again in the
    row's log-sum-exp (fp32), which enters the accumulated weights; the prefix's exponents are
    formed by one FMA.  The scale's own rounding (2^-24) times the difference of two logits
    that both count (under 2^5) is below 2^-18."""
    for sign, own in ((1, 0), (1, 3), (1, -3), (-1, 2)):
        c = make(cuda_dev, n_seq, 1, 8, 2, D, 16, [(5 * s) % 40 for s in range(n_seq)], 700, 20, poison=False)
        c = large_logits(c, n_seq, D, sign, own)
        if sign < 0:                             # from -3e5 to 3e5 within a row
            c["pk"][350:] = -c["pk"][350:]
        d, cache = on(cuda_dev, c, crs)
        mo = d["mass"].clone()
        O, lse = cache.attend(d["q"], d["pk"], d["pv"], scale=scale, out_dtype=out_dtype, mass_out=mo)
        torch.cuda.synchronize()
        assert crs.get_device_error() == 0
        eO, el, em, A = ref.attend(c["q"], c["k"], c["v"], c["table"], c["seq_len"], c["cap"], None, c["pk"], c["pv"],
                                   scale=scale, mass=c["mass"])
        z = 2.0 * float(el.abs().max()) * 2.0 ** -24
        half = 0.0 if out_dtype == torch.float32 else 2.0 ** -8
        o = O.double().cpu()
        tol = A * (2.0 ** -14 + 2.0 ** -17 + z + half) + eO.abs() * (half or 2.0 ** -24)
        assert torch.isfinite(o).all() and ((o - eO).abs() <= tol).all(), (sign, own)
        assert ((lse.double().cpu() - el).abs() <= el.abs() * 2.0 ** -22 + 2.0 ** -15).all()
        got, add = mo.double().cpu(), (em - c["mass"].double()).abs()
        for s in range(n_seq):
            t = int(c["seq_len"][s]) + 1
            assert ((got - em).abs() <= add * (2.0 ** -14 + z) + em.abs() * 2.0 ** -21)[s, :, :t].all()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,n_seq", [(64, 20), (128, 20), (128, 70)])
@pytest.mark.parametrize("column", range(0, 16, 3))
def test_far_keys_of_the_prefix_add_nothing(crs, cuda_dev, out_dtype, D, n_seq, column):
    """Keys some 500 to 1000 log2 units below the others, whose values are 2^126: their weight is
    0 in any 32-bit form, so nothing of them may reach the output."""
    c = make(cuda_dev, n_seq, 1, 8, 2, D, 16, [s % 9 for s in range(n_seq)], 400, 22, poison=False)
    c["q"] = torch.full_like(c["q"], 4.0)
    c["k"], c["pk"] = c["k"] * 0.125, c["pk"] * 0.125
    c["pk"][column::16] = -12.0
    c["pv"][column::16] = 2.0 ** 126
    check(crs, cuda_dev, c, out_dtype, scale=0.125, with_mass=False)


def test_weights_of_accepted_drafts_only(crs, cuda_dev):
    """Drafts are attended without weights, then once more as far as they were accepted: outputs
    of the accepted tokens come again, and the weights are those of these tokens alone."""
    n_tok, lens = 4, [0, 9, 40, 63, 100]
    c = make(cuda_dev, 5, n_tok, 8, 2, 128, 16, lens, 90, 23)
    d, cache = on(cuda_dev, c, crs)
    O, lse = cache.attend(d["q"], d["pk"], d["pv"])
    assert torch.equal(cache.mass.cpu(), c["mass"])
    acc = torch.tensor([0, 1, 4, 2, 3], dtype=torch.int32)
    O2, lse2 = cache.attend(d["q"], d["pk"], d["pv"], n_new=acc.to(cuda_dev), mass_out=cache.mass)
    _, _, em, A = ref.attend(c["q"], c["k"], c["v"], c["table"], c["seq_len"], c["cap"], acc, c["pk"], c["pv"],
                             mass=c["mass"])
    for s in range(5):
        n, t = int(acc[s]), lens[s] + int(acc[s])
        # the slots' tiles may be cut elsewhere: twice the f32 tolerance above
        assert ((O[s, :n] - O2[s, :n]).double().cpu().abs() <= 2 * TOL_F32 * A[s, :n] + 1e-30).all()
        tol = (em - c["mass"].double()).abs() * 2.0 ** -14 + em.abs() * 2.0 ** -21
        assert ((cache.mass.double().cpu() - em).abs() <= tol)[s, :, :t].all()
        assert torch.equal(cache.mass[s, :, t:].cpu(), c["mass"][s, :, t:])
    cache.commit(acc.to(cuda_dev), n_tok=n_tok)
    assert cache.seq_len.tolist() == [l + int(a) for l, a in zip(lens, acc)]
    assert crs.get_device_error() == 0
