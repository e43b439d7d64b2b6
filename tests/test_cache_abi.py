"""Refusals of the decode-cache calls, on the host, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
OK = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def by(x):
    return ctypes.byref(x)


def rope_call(crs, p, n_tok=4, heads=2, dtype=1, x=OK, xs=None, pos=OK, f=OK, y=ctypes.c_void_p(0x20000), ys=None):
    row = heads * p.D
    return crs.lib().crs_rope(by(p), n_tok, heads, dtype, x, row if xs is None else xs, pos, f, y,
                              row if ys is None else ys, None)


def test_rope_refusals(crs):
    R = crs.RopeParams
    good = R(64, 0, 64, 0, 0, 1.0)
    assert crs.lib().crs_rope(None, 1, 1, 1, OK, 64, OK, OK, OK, 64, None) == INVALID
    for p in (R(0, 0, 0, 0, 0, 1.0), R(64, -2, 32, 0, 0, 1.0), R(64, 0, 31, 0, 0, 1.0), R(64, 40, 32, 0, 0, 1.0),
              R(64, 0, -2, 0, 0, 1.0)):
        assert rope_call(crs, p) == INVALID
    assert rope_call(crs, R(2048, 0, 64, 0, 0, 1.0)) == UNSUPPORTED
    assert rope_call(crs, good, n_tok=-1) == INVALID
    assert rope_call(crs, good, heads=0, xs=64, ys=64) == INVALID
    assert rope_call(crs, good, dtype=2) == INVALID
    assert rope_call(crs, good, n_tok=0, x=None) == 0                     # nothing to do
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(f=None)):
        assert rope_call(crs, good, **kw) == INVALID
    assert rope_call(crs, good, xs=127) == INVALID                        # rows overlap
    assert rope_call(crs, good, ys=64) == INVALID
    assert rope_call(crs, good, x=OK, y=OK, xs=128, ys=256) == INVALID    # in place wants one stride
    assert rope_call(crs, good, x=ctypes.c_void_p(0x10001)) == INVALID


CACHE = dict(n_seq=2, n_kv=2, D=128, page_size=16, max_pages=4, n_pages=8, cap=60)


def cache(crs, **kw):
    return crs.CacheParams(**{**CACHE, **kw})


def state(crs, **kw):
    names = [n for n, _ in crs.CacheState._fields_]
    return crs.CacheState(**{**{n: 0x10000 for n in names}, **kw})


BAD_CACHES = [(dict(n_seq=0), INVALID), (dict(n_kv=0), INVALID), (dict(page_size=0), INVALID),
              (dict(max_pages=0), INVALID), (dict(n_pages=0), INVALID), (dict(cap=0), INVALID),
              (dict(D=96), UNSUPPORTED), (dict(n_seq=5000), UNSUPPORTED), (dict(cap=65), UNSUPPORTED),
              (dict(page_size=1 << 16, n_pages=1 << 16), UNSUPPORTED)]
BAD_STATES = ["k_pool", "v_pool", "block_table", "seq_len", "next_pos"]


def append_call(crs, p, st, r=None, f=None, n_tok=1, k=OK, ks=256, v=OK, vs=256, q=None, qs=512, n_q=4, qo=OK):
    return crs.lib().crs_cache_append(by(p), by(st), None if r is None else by(r), f, n_tok, None, k, ks, v, vs, q, qs,
                                      n_q, qo, None)


def test_append_and_commit_refusals(crs):
    st = state(crs)
    for kw, want in BAD_CACHES:
        assert append_call(crs, cache(crs, **kw), st) == want
        assert crs.lib().crs_cache_commit(by(cache(crs, **kw)), by(st), 1, None, None) == want
    p = cache(crs)
    for n in BAD_STATES:
        assert append_call(crs, p, state(crs, **{n: None})) == INVALID
        assert crs.lib().crs_cache_commit(by(p), by(state(crs, **{n: None})), 1, None, None) == INVALID
    assert append_call(crs, p, state(crs, k_pool=0x10008)) == INVALID
    assert crs.lib().crs_cache_commit(by(p), by(st), -1, None, None) == INVALID
    R = crs.RopeParams
    for kw in (dict(n_tok=0), dict(k=None), dict(v=None), dict(k=ODD), dict(ks=255), dict(ks=260), dict(vs=128),
               dict(q=OK, qo=None), dict(q=OK, n_q=0), dict(q=OK, qs=511), dict(q=ODD), dict(q=OK, qo=ODD),
               dict(r=R(64, 0, 64, 0, 0, 1.0), f=OK), dict(r=R(128, 0, 128, 0, 0, 1.0), f=None)):
        assert append_call(crs, p, st, **kw) == INVALID
    assert append_call(crs, p, st, r=R(128, 4, 64, 0, 0, 1.0), f=OK) == UNSUPPORTED
    assert append_call(crs, p, st, r=R(128, 0, 24, 0, 0, 1.0), f=OK) == UNSUPPORTED


def attn(crs, c=None, **kw):
    d = dict(n_q=4, n_tok=1, prefix_len=100, out_dtype=0, want_mass=0, scale=0.1, decay=1.0)
    return crs.CacheAttnParams(c if c is not None else cache(crs), **{**d, **kw})


def attn_call(crs, p, st=None, Q=OK, pk=OK, pv=OK, O=OK, mass=None, ws=None, ws_bytes=0):
    return crs.lib().crs_cache_attn(by(p), by(st if st is not None else state(crs)), Q, None, pk, pv, O, None, mass, ws,
                                    ws_bytes, None)


def test_attention_refusals(crs):
    for kw, want in BAD_CACHES:
        p = attn(crs, cache(crs, **kw))
        assert attn_call(crs, p) == want
        assert crs.lib().crs_cache_attn_workspace_size(by(p)) == 0
    for kw, want in ((dict(n_q=0), INVALID), (dict(n_tok=0), INVALID), (dict(prefix_len=-1), INVALID),
                     (dict(out_dtype=7), INVALID), (dict(n_q=3), UNSUPPORTED), (dict(n_q=130), UNSUPPORTED),
                     (dict(n_tok=600), UNSUPPORTED)):
        assert attn_call(crs, attn(crs, **kw)) == want
    huge = cache(crs, n_seq=4096, page_size=1 << 20, max_pages=2000, n_pages=1, cap=2000 << 20)
    assert attn_call(crs, attn(crs, huge)) == UNSUPPORTED                 # units past 32 bits
    p = attn(crs)
    for n in BAD_STATES:
        assert attn_call(crs, p, state(crs, **{n: None})) == INVALID
    for kw in (dict(Q=None), dict(O=None), dict(pk=None), dict(pv=None), dict(Q=ODD), dict(O=ODD), dict(pk=ODD)):
        assert attn_call(crs, p, **kw) == INVALID
    m = attn(crs, want_mass=1)
    assert attn_call(crs, m) == INVALID
    assert attn_call(crs, m, state(crs, mass=None), mass=OK) == INVALID
    need = crs.lib().crs_cache_attn_workspace_size(by(p))
    assert need > 0
    assert attn_call(crs, p) == WORKSPACE
    assert attn_call(crs, p, ws=OK, ws_bytes=need - 1) == WORKSPACE
    assert attn_call(crs, p, ws=ODD, ws_bytes=need) == INVALID


def test_select_and_evict_refusals(crs):
    L = crs.lib()
    S = crs.MassSelectParams
    assert L.crs_mass_select(None, *([OK] * 6), None) == INVALID
    for p in (S(0, 1, 8, 4, 0, 0), S(1, 0, 8, 4, 0, 0), S(1, 1, 0, 1, 0, 0), S(1, 1, 8, 0, 0, 0), S(1, 1, 8, 9, 0, 0),
              S(1, 1, 8, 4, 0, -1)):
        assert L.crs_mass_select(by(p), *([OK] * 6), None) == INVALID
    p = S(1, 1, 8, 4, 0, 0)
    for i in (0, 2, 4, 5):                                                # mass, seq_len, idx, count
        args = [OK] * 6
        args[i] = None
        assert L.crs_mass_select(by(p), *args, None) == INVALID
    assert L.crs_mass_select(by(p), OK, OK, OK, None, OK, OK, None) == INVALID     # pos without next_pos
    for kw, want in BAD_CACHES:
        assert L.crs_cache_evict(by(cache(crs, **kw)), by(state(crs)), 4, OK, OK, None) == want
    c = cache(crs)
    for n in BAD_STATES:
        assert L.crs_cache_evict(by(c), by(state(crs, **{n: None})), 4, OK, OK, None) == INVALID
    assert L.crs_cache_evict(by(c), by(state(crs)), 0, OK, OK, None) == INVALID
    assert L.crs_cache_evict(by(c), by(state(crs)), 4, None, OK, None) == INVALID
    assert L.crs_cache_evict(by(c), by(state(crs)), 4, OK, None, None) == INVALID


def test_binding_refuses_cpu_tensors_and_bad_frequencies(crs):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        crs.rope(x, torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        crs.mass_select(torch.zeros(1, 1, 8), torch.zeros(1, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        crs.KvCache.empty(1, 1, 16, device="cpu")
    for bad in (dict(rot_dim=3), dict(rot_dim=8, base=1.0), dict(rot_dim=8, factor=0.0),
                dict(rot_dim=8, scaling="other")):
        with pytest.raises(ValueError):
            crs.rope_inv_freq(**{"device": "cpu", **bad})


def test_row_strides(crs):
    """Token rows may be slices of a wider projection; anything else is refused."""
    dev = torch.zeros(1).get_device()
    t = torch.zeros(3, 5, 8, 64, dtype=torch.bfloat16)
    rows = lambda v: crs._rows(v, "v", torch.bfloat16, v.shape, dev)  # noqa: E731
    assert rows(t) == 8 * 64
    assert rows(t[:, :, 2:4]) == 8 * 64
    assert rows(t[:, :1, 2:4]) == 5 * 8 * 64                              # one token of each sequence
    assert rows(t[:1, :, 2:4]) == 8 * 64
    assert rows(t[:1, :1, 2:4]) == 2 * 64                                 # a single row
    with pytest.raises(ValueError):
        rows(t[:, :2, 2:4])                                               # unevenly spaced
    with pytest.raises(ValueError):
        rows(t[..., :32])                                                 # heads not dense
    with pytest.raises(ValueError):
        rows(t.transpose(1, 2))
    with pytest.raises(ValueError):
        rows(t[:, :1].expand(3, 5, 8, 64))                                # stride 0


def test_select_refuses_lengths_as_output(crs):
    """The heads of a sequence run side by side: a count written over the lengths (or the next
    positions) would be read by the others."""
    L, S = crs.lib(), crs.MassSelectParams
    at = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6)]           # mass, pos, seq_len, next_pos, idx, count
    for shared in ((5, 2), (5, 3), (4, 1), (4, 0), (4, 2), (4, 3), (5, 4)):
        args = list(at)
        args[shared[0]] = args[shared[1]]
        assert L.crs_mass_select(by(S(2, 2, 8, 4, 0, 1)), *args, None) == INVALID, shared
