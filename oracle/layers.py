"""fp64 CPU oracle of the operators around a GDN layer: attention of new tokens
over a paged cache, cache write, eviction, block norms.

TEST INFRASTRUCTURE, like the rest of this folder.  Everything is written from
the definitions, one row and one token at a time where that is plainest, on
numpy arrays; it shares no code with the library.
"""
from __future__ import annotations

import numpy as np


def token_row(pool, table_row, pos, h):
    """The (token, head) row at position pos of a table row; None on a bad page."""
    page = pool.shape[2]
    pg = int(table_row[pos // page])
    if not 0 <= pg < pool.shape[0]:
        return None
    return pool[pg, h, pos % page].astype(np.float64)


def gather(pool, table_row, n, h):
    """Rows of the first n positions that lie on a page: their positions, [m][d]."""
    pos, rows = [], []
    for p in range(n):
        x = token_row(pool, table_row, p, h)
        if x is not None:
            pos.append(p)
            rows.append(x)
    return np.array(pos, dtype=np.int64), np.array(rows).reshape(len(rows), pool.shape[3])


def clamp(n, hi):
    return max(0, min(int(n), hi))


def paged_attention(q, k_pool, v_pool, table, lengths, beam=None, scale=None, mass=None):
    """Returns o [R][W][H_q][d], lse [R][W][H_q], drawn [R][H_kv][row_pages page]
    (the weights added up, on top of mass), spread [R][W][H_q][d] = sum p |v|
    (what tolerances scale with)."""
    q = np.asarray(q, dtype=np.float64)
    R, W, H_q, d = q.shape
    H, page = k_pool.shape[1], k_pool.shape[2]
    G, cap = H_q // H, table.shape[1] * page
    scale = d ** -0.5 if scale is None else scale
    o, spread = np.zeros((R, W, H_q, d)), np.zeros((R, W, H_q, d))
    lse = np.full((R, W, H_q), -np.inf)
    drawn = np.zeros((R, H, cap)) if mass is None else np.asarray(mass, dtype=np.float64).copy()
    for r in range(R):
        for h in range(H):
            n = clamp(lengths[r], cap)
            pos, k = gather(k_pool, table[r], n, h)
            _, v = gather(v_pool, table[r], n, h)
            for w in range(W):
                kk, vv = k, v
                if beam is not None:
                    bk, bv, bt, bl = beam
                    nb = clamp(bl[r][w], bt.shape[2] * bk.shape[2])
                    kk = np.concatenate([k, gather(bk, bt[r][w], nb, h)[1]])
                    vv = np.concatenate([v, gather(bv, bt[r][w], nb, h)[1]])
                if not len(kk):
                    continue
                for g in range(G):
                    s = kk @ q[r, w, h * G + g] * scale
                    top = s.max()
                    e = np.exp(s - top)
                    p = e / e.sum()
                    o[r, w, h * G + g] = p @ vv
                    spread[r, w, h * G + g] = p @ np.abs(vv)
                    lse[r, w, h * G + g] = top + np.log(e.sum())
                    drawn[r, h, pos] += p[:len(pos)]
    return o, lse, drawn, spread


def cache_write(k, pool, table, start, counts=None):
    """A copy of pool with the tokens of k [B][n][H][d] written (one of k, v at a time)."""
    pool = pool.copy()
    pages, H, page, d = pool.shape
    for b in range(k.shape[0]):
        n = k.shape[1] if counts is None else clamp(counts[b], k.shape[1])
        for i in range(n):
            pos = int(start[b]) + i
            if not 0 <= pos < table.shape[1] * page:
                continue
            pg = int(table[b, pos // page])
            if 0 <= pg < pages:
                pool[pg, :, pos % page] = k[b, i]
    return pool


def kept_positions(weights, length, keep, recent):
    """The positions of one (request, head) that stay, in order."""
    n = min(length, keep)
    last = min(recent, n)
    free = length - last

    def order(p):
        w = float(weights[p])
        return (1, 0.0, p) if np.isnan(w) else (0, -w, p)

    best = sorted(range(free), key=order)[: n - last]
    return sorted(best) + list(range(free, length))


def cache_evict(k_pool, v_pool, table, lengths, mass, keep, recent, dst_k, dst_v, dst_table, dst_mass):
    """Copies of (dst_k, dst_v, dst_mass) after the eviction, the new lengths and kept [R][H][keep]."""
    dst_k, dst_v, dst_mass = dst_k.copy(), dst_v.copy(), dst_mass.copy()
    R, H, cap = mass.shape
    page = k_pool.shape[2]
    new = np.zeros((R,), np.int32)
    kept = np.full((R, H, keep), -1, np.int32)
    for r in range(R):
        length = clamp(lengths[r], cap)
        new[r] = min(length, keep)
        for h in range(H):
            for j, p in enumerate(kept_positions(mass[r, h], length, keep, recent)):
                kept[r, h, j] = p
                dst_mass[r, h, j] = mass[r, h, p]
                to = int(dst_table[r, j // page])
                if not 0 <= to < dst_k.shape[0]:
                    continue
                for src, dst in ((k_pool, dst_k), (v_pool, dst_v)):
                    pg = int(table[r, p // page])
                    ok = 0 <= pg < src.shape[0]
                    dst[to, h, j % page] = src[pg, h, p % page] if ok else 0
    return dst_k, dst_v, dst_mass, new, kept


def block_norm(y=None, x=None, gate=None, act="none", w_post=None, scale=None, alpha=1.0, w_pre=None, eps=1e-6):
    """(x', n') in fp64; n' None without w_pre."""
    if y is None:
        out = np.asarray(x, dtype=np.float64)
    else:
        u = np.asarray(y, dtype=np.float64).copy()
        N, D = u.shape
        if w_post is not None:
            g = len(w_post)
            for c in range(0, D, g):
                part = u[:, c:c + g]
                u[:, c:c + g] = part / np.sqrt((part ** 2).mean(1, keepdims=True) + eps) * np.asarray(w_post, np.float64)
        if gate is not None:
            z = np.asarray(gate, dtype=np.float64)
            sig = 0.5 * (1.0 + np.tanh(0.5 * z))
            u *= {"sigmoid": sig, "silu": z * sig}[act]
        u *= alpha
        if scale is not None:
            u *= np.asarray(scale, np.float64)
        out = u if x is None else np.asarray(x, dtype=np.float64) + u
    if w_pre is None:
        return out, None
    return out, out / np.sqrt((out ** 2).mean(1, keepdims=True) + eps) * np.asarray(w_pre, np.float64)
