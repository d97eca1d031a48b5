"""Oracle of the prompt side of the cache (plain Python and numpy, float64 for
the arithmetic). Test infrastructure only; shares no code with the library.
Requests, pages and tokens are walked one by one, as the definitions read.
"""
from __future__ import annotations

import math

import numpy as np


def plan(ctx, new, held, free, count, table, page, T):
    """One request after another. Returns a dict of the state and rows after; `left` lists the requests that found no
    room, `bad` those that are not valid. A row whose page is not one of the pool has slot -1."""
    B, cols = table.shape
    table, held = table.copy(), [int(x) for x in held]
    want_pages = want_rows = given = rows = 0
    q_start, kv_len, granted, pos, slot, left, bad = [0], [], [], [], [], [], []
    for b in range(B):
        c, n, h = int(ctx[b]), int(new[b]), held[b]
        take = 0
        if c < 0 or n < 0 or not 0 <= h <= cols or c > h * page or c + n > cols * page:
            bad.append(b)
        else:
            need = max(0, math.ceil((c + n) / page) - h) if n else 0
            want_pages += need
            want_rows += n
            if (need and want_pages > count) or (n and want_rows > T):
                left.append(b)
            else:
                take = n
                for i in range(need):
                    table[b, h + i] = free[count - 1 - given]
                    given += 1
                held[b] = h + need
        for i in range(take):
            pos.append(c + i)
            p = int(table[b, (c + i) // page])
            slot.append(p * page + (c + i) % page if 0 <= p < len(free) else -1)
        rows += take
        q_start.append(rows)
        kv_len.append(min(max(c, 0), cols * page) + take)
        granted.append(take)
    pad = [-1] * (T - rows)
    i32 = lambda x: np.array(x, np.int32)  # noqa: E731
    return dict(table=table, held=i32(held), count=count - given, q_start=i32(q_start), kv_len=i32(kv_len),
                granted=i32(granted), pos=i32(pos + pad), slot=i32(slot + pad), left=left, bad=bad)


def release(done, held, free, count, table):
    free, held = free.copy(), held.copy()
    for b in range(len(done)):
        if done[b]:
            for i in range(int(held[b])):
                free[count] = table[b, i]
                count += 1
            held[b] = 0
    return free, count, held


def norm_rope(x, w, pos, inv_freq, rot, interleaved, mscale, eps):
    """x [T, H, D] float64 -> (result, the magnitudes |a| + |b| that meet in each element); w None = no norm."""
    x = x.astype(np.float64).copy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    mag = np.abs(x)
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = pos.astype(np.float64) * inv_freq[i]
        c, s = (np.cos(ang) * mscale)[:, None], (np.sin(ang) * mscale)[:, None]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
        mag[..., a] = mag[..., b] = (np.abs(xa) + np.abs(xb)) * abs(mscale)
    return x, mag


def chunk_attention(q, k, v, q_start, kv_len, table, page, scale):
    """q [T, Hq, D], pages k, v [pages, Hkv, page, D], all float64. Returns out, lse and, for the bounds of a kernel's
    error, per row and head: sum p|v| [.., D], the largest |q|.|k| scale, the largest |s| and the number of keys.
    A key takes part when its page is one of the pool."""
    T, Hq, D = q.shape
    pages, Hkv = k.shape[:2]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    absv, prod, smax, keys = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        n, L = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        if n == 0 or L == 0:
            continue
        j = np.arange(L)
        p = table[b, j // page]
        there = (p >= 0) & (p < pages)
        p = np.where(there, p, 0)
        for h in range(Hkv):
            kk = np.where(there[:, None], k[p, h, j % page], 0.0)
            vv = np.where(there[:, None], v[p, h, j % page], 0.0)
            for g in range(G):
                hq = h * G + g
                rows = np.arange(q_start[b], q_start[b + 1])
                s = q[rows, hq] @ kk.T * scale
                see = there[None, :] & (j[None, :] <= (L - n + np.arange(n))[:, None])
                ab = np.where(see, np.abs(q[rows, hq]) @ np.abs(kk).T * scale, 0.0)
                s = np.where(see, s, -np.inf)
                m = s.max(1)
                some = np.isfinite(m)
                w = np.exp(s - np.where(some, m, 0.0)[:, None])
                l = w.sum(1)
                w = w / np.where(l > 0, l, 1.0)[:, None]
                out[rows, hq] = w @ vv
                absv[rows, hq] = w @ np.abs(vv)
                with np.errstate(divide="ignore"):
                    lse[rows, hq] = np.where(some, m + np.log(l), -np.inf)
                prod[rows, hq], keys[rows, hq] = ab.max(1), see.sum(1)
                smax[rows, hq] = np.where(see, np.abs(s), 0.0).max(1)
    return out, lse, absv, prod, smax, keys


def fill(pk, pv, table, page, kv_len, dense, head, sparse, take=None):
    """The tiers after kv_len[b] appends to empty ones, through the append oracle, token by token. Requests that are
    not taken keep what they have. pk, pv [pages, Hkv, page, D]; returns (dense, head, sparse, dropped counts)."""
    from . import Tier, append

    H = pk.shape[1]
    out = [dense.k.copy(), dense.v.copy(), dense.len.copy(), head.copy(), sparse.k.copy(), sparse.v.copy(),
           sparse.len.copy(), np.zeros(len(head), np.int32)]
    for b in range(len(kv_len)):
        if take is not None and not take[b]:
            continue
        u = slice(b * H, b * H + H)
        d = Tier(out[0][b:b + 1], out[1][b:b + 1], np.zeros(H, np.int32))
        s = Tier(out[4][b:b + 1], out[5][b:b + 1], np.zeros(H, np.int32))
        hd, lost = np.zeros(H, np.int32), np.zeros(H, np.int32)
        for t in range(int(kv_len[b])):
            p = int(table[b, t // page])
            ok = 0 <= p < len(pk)
            kn = pk[p, :, t % page] if ok else np.zeros_like(pk[0, :, 0])
            vn = pv[p, :, t % page] if ok else np.zeros_like(pv[0, :, 0])
            d, hd, s, dr = append(kn[None], vn[None], d, hd, s)
            lost += dr
        for i, x in ((0, d.k), (1, d.v), (4, s.k), (5, s.v)):
            out[i][b:b + 1] = x
        out[2][u], out[3][u], out[6][u], out[7][u] = d.len, hd, s.len, lost
    return Tier(out[0], out[1], out[2]), out[3], Tier(out[4], out[5], out[6]), out[7]
