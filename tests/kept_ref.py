"""fp64 references of the cache-eviction operators, slot by slot, and inputs for their tests."""
import math

import numpy as np
import torch

import oracle.bifocal_ref as R
import seeded_inputs as si

THETA = 1e6


def page_table(lens, page, gen, spare=2):
    """Block table over shuffled pages (unused entries -1), and the pages in all."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen).int()
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, pages


def row_of(table, page, b, slot):
    return int(table[b, slot // page]) * page + slot % page


def rows_of(table, page, b, n):
    return np.array([row_of(table, page, b, s) for s in range(n)], dtype=np.int64)


def far(pos, G, mode):
    pos = np.asarray(pos, dtype=np.float64)
    return pos / G if mode == si.FREQ_INTERP else np.floor(pos / G)


def rotate(x, pos):
    """x [n, D] at positions pos [n] (real numbers)."""
    return R.rope_rotate(np.asarray(x, dtype=np.float64), np.asarray(pos, dtype=np.float64), R.rope_omega(x.shape[-1], THETA))


def decode_kept(q, kc, vc, pos, now, w0, wp, mode, window=False):
    """One sequence and kv head. q [g, D] raw; kc / vc [n, D] as the cache holds them; pos [n]. Returns out [g, D],
    lse [g], the weights [n] summed over the group, and sum_j p_j |v_j| [g, D]."""
    G = R.dynamic_factor(now + 1, wp)
    D = q.shape[1]
    here = np.full(len(q), float(now))
    raw = rotate(kc, -np.asarray(pos, dtype=np.float64))
    s_near = rotate(q, here) @ np.asarray(kc, dtype=np.float64).T
    s_far = rotate(q, far(here, G, mode)) @ rotate(raw, far(pos, G, mode)).T
    near = (now - np.asarray(pos, dtype=np.int64)) < w0
    s = np.where(near, s_near, -np.inf if window else s_far) / math.sqrt(D)
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    p = e / e.sum(1, keepdims=True)
    return p @ vc, (m + np.log(e.sum(1, keepdims=True)))[:, 0], p.sum(0), p @ np.abs(vc)


def choose(pos, weight, newest, budget, recent, sink):
    """Slots kept, ascending: protected positions, then larger weights (NaN as -inf), then lower slots."""
    def rank(s):
        if pos[s] < sink or pos[s] > newest - recent:
            return (0, 0.0, s)
        w = weight[s]
        return (1, math.inf if w != w else -float(w), s)
    return sorted(sorted(range(len(pos)), key=rank)[:budget])


def moves(kept, n, in_place):
    """(source slot, destination slot) pairs."""
    if not in_place:
        return list(zip(kept, range(len(kept))))
    m = len(kept)
    holes = sorted(set(range(min(m, n))) - set(kept))
    return list(zip([s for s in kept if s >= m], holes))
