"""Plain 64-bit forms of the decode-cache operators, on the CPU, written from their
definitions with explicit loops over sequences and heads."""
import math

import torch


def rope(x, pos, inv_freq, rot_begin=0, interleaved=False, mscale=1.0, inverse=False):
    """x [..., heads, D] (any float type), pos [...] -> float64."""
    y = x.double().clone()
    half = inv_freq.numel()
    ang = pos.double()[..., None, None] * inv_freq.double()
    c, s = torch.cos(ang) * mscale, torch.sin(ang) * mscale
    if inverse:
        s = -s
    j = torch.arange(half)
    ia, ib = (rot_begin + 2 * j, rot_begin + 2 * j + 1) if interleaved else (rot_begin + j, rot_begin + half + j)
    a, b = x.double()[..., ia], x.double()[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def n_used(n_new, n_tok, seq_len, cap):
    """Tokens of each sequence that count."""
    n_seq = len(seq_len)
    asked = [n_tok] * n_seq if n_new is None else [min(max(int(v), 0), n_tok) for v in n_new]
    return [min(a, cap - int(l)) for a, l in zip(asked, seq_len)]


def slots(pool, table, s, page, total):
    """[total, n_kv, D] float64: the sequence's slots in order."""
    rows = [pool[int(table[s, j // page]), j % page] for j in range(total)]
    return torch.stack(rows).double() if rows else torch.zeros((0,) + tuple(pool.shape[2:]), dtype=torch.float64)


def attend(q, k_pool, v_pool, table, seq_len, cap, n_new=None, pk=None, pv=None, scale=None, mass=None, decay=1.0):
    """-> (O [n_seq, n_tok, n_q, D], lse, mass_out, sum_abs) float64; sum_abs [like O] is
    sum_j p_j |v_j|, which scales the rounding of the weights."""
    n_seq, n_tok, n_q, D = q.shape
    page, n_kv = k_pool.shape[1], k_pool.shape[2]
    G = n_q // n_kv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    O = torch.zeros(q.shape, dtype=torch.float64)
    A = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((n_seq, n_tok, n_q), -math.inf, dtype=torch.float64)
    mo = None if mass is None else mass.double().clone()
    used = n_used(n_new, n_tok, seq_len, cap)
    plen = 0 if pk is None else pk.shape[0]
    for s in range(n_seq):
        total = int(seq_len[s]) + used[s]
        ks, vs = slots(k_pool, table, s, page, total), slots(v_pool, table, s, page, total)
        if mo is not None:
            mo[s, :, :total] *= decay
        for i in range(used[s]):
            see = int(seq_len[s]) + i + 1
            for hq in range(n_q):
                h = hq // G
                K, V = ks[:see, h], vs[:see, h]
                if plen:
                    K, V = torch.cat([pk[:, h].double(), K]), torch.cat([pv[:, h].double(), V])
                z = (K @ q[s, i, hq].double()) * scale
                lse[s, i, hq] = torch.logsumexp(z, 0)
                p = torch.exp(z - lse[s, i, hq])
                O[s, i, hq] = p @ V
                A[s, i, hq] = p @ V.abs()
                if mo is not None:
                    mo[s, h, :see] += p[plen:]
    return O, lse, mo, A


def select(mass, seq_len, keep, pos=None, next_pos=None, sink_end=0, window=0):
    n_seq, n_kv, cap = mass.shape
    idx = torch.full((n_seq, n_kv, keep), -1, dtype=torch.int32)
    count = torch.zeros(n_seq, dtype=torch.int32)
    for s in range(n_seq):
        n = min(max(int(seq_len[s]), 0), cap)
        k = min(keep, n)
        count[s] = k
        for h in range(n_kv):
            def rank(j):
                m = float(mass[s, h, j])
                fixed = pos is not None and (int(pos[s, h, j]) < sink_end or
                                             int(pos[s, h, j]) >= int(next_pos[s]) - window)
                if fixed:
                    return (0, 0.0, j)
                return (2, 0.0, j) if math.isnan(m) else (1, -m, j)
            best = sorted(range(n), key=rank)[:k]
            idx[s, h, :k] = torch.tensor(sorted(best), dtype=torch.int32)
    return idx, count


def evict(k_pool, v_pool, table, pos, mass, idx, count):
    """Copies with the kept rows moved, by the rule: r-th kept slot >= n to the r-th free one < n."""
    k, v, pos, mass = k_pool.clone(), v_pool.clone(), pos.clone(), mass.clone()
    page, n_kv = k.shape[1], k.shape[2]
    for s in range(idx.shape[0]):
        n = int(count[s])
        for h in range(n_kv):
            kept = [int(x) for x in idx[s, h, :n]]
            src = [x for x in kept if x >= n]
            dst = [x for x in range(n) if x not in set(kept)]
            for a, b in zip(src, dst):
                pa, pb = int(table[s, a // page]), int(table[s, b // page])
                k[pb, b % page, h] = k_pool[pa, a % page, h]
                v[pb, b % page, h] = v_pool[pa, a % page, h]
                pos[s, h, b] = pos[s, h, a]
                mass[s, h, b] = mass[s, h, a]
    return k, v, pos, mass
