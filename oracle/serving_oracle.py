"""Float64 CPU oracle of the paged serving calls, request by request.

plan_pages and verify_draft follow the definitions in the C header one request at a
time, with Python integers and float64; paged_attention gathers a request's rows page
by page and takes the softmax of every new token by itself, from the absorbed query.
None of it shares code or order of work with the kernels.
"""
from __future__ import annotations

import numpy as np


def plan_pages(page, num_pages, kept, n_new, held, free, count, table, room):
    """One step of the page plan.  Returns a dict of the outputs, as lists."""
    B, width = len(kept), len(table[0]) if len(table) else 0
    table = [list(r) for r in table]
    free = list(free)
    goal = [-(-(k + n) // page) for k, n in zip(kept, n_new)]
    bad = [k < 0 or n < 0 or h < 0 or h > width or t > width or k > h * page
           for k, n, h, t in zip(kept, n_new, held, goal)]
    fits, asked = [], 0
    for b in range(B):
        if not bad[b]:
            asked += n_new[b]
        fits.append(not bad[b] and asked <= room)
    returned = sum(max(held[b] - goal[b], 0) for b in range(B) if fits[b])
    broken = count < 0 or count + returned > num_pages
    top = count + returned
    granted, wanted = [], 0
    for b in range(B):
        need = max(goal[b] - held[b], 0) if fits[b] else 0
        wanted += need
        granted.append(fits[b] and not broken and (need == 0 or wanted <= top))
    err = (1 if any(bad) or broken else 0) | (4 if any(not g and not x for g, x in zip(granted, bad)) else 0)
    for b in range(B):
        if granted[b]:
            for t in range(goal[b], held[b]):
                free[count] = table[b][t]
                count += 1
    out = dict(held=[], q_start=[0], seq_len=[], n_granted=[], slot=[], pos=[])
    for b in range(B):
        if granted[b]:
            for t in range(held[b], goal[b]):
                count -= 1
                table[b][t] = free[count]
            for p in range(kept[b], kept[b] + n_new[b]):
                pg = table[b][p // page]
                ok = 0 <= pg < num_pages
                err |= 0 if ok else 1
                out["slot"].append(pg * page + p % page if ok else -1)
                out["pos"].append(p)
        out["held"].append(goal[b] if granted[b] else held[b])
        out["n_granted"].append(n_new[b] if granted[b] else 0)
        out["seq_len"].append((0 if bad[b] else kept[b]) + out["n_granted"][b])
        out["q_start"].append(len(out["slot"]))
    fill = [-1] * (room - len(out["slot"]))
    out["slot"] += fill
    out["pos"] += fill
    out.update(free=free, count=count, table=table, err=err)
    return out


def paged_attention(q_abs, V, kr, table, page, q_start, seq_len, G):
    """Outputs, natural-log lse and sum of p |v| of every query row; rows of no request
    are NaN.  q_abs [N, H, d_h + d_r] in base-2 units, V [slots, G, d_h], kr [slots, d_r].
    A page outside the cache reads as zeros."""
    q_abs, V, kr = (np.asarray(x, dtype=np.float64) for x in (q_abs, V, kr))
    N, H, _ = q_abs.shape
    d_h, hpr = V.shape[2], H // G
    out = np.full((N, H, d_h), np.nan)
    mag = np.full((N, H, d_h), np.nan)
    lse = np.full((N, H), np.nan)
    for b in range(len(seq_len)):
        L, r0, n = int(seq_len[b]), int(q_start[b]), int(q_start[b + 1] - q_start[b])
        if n == 0:
            continue
        v, k = np.zeros((L, G, d_h)), np.zeros((L, kr.shape[1]))
        for t in range(L):
            pg = int(table[b][t // page]) if t // page < len(table[b]) else -1
            if 0 <= pg < V.shape[0] // page:
                v[t], k[t] = V[pg * page + t % page], kr[pg * page + t % page]
        for i in range(n):
            keys = max(0, L - n + i + 1)
            for h in range(H):
                if keys == 0:
                    out[r0 + i, h], mag[r0 + i, h], lse[r0 + i, h] = 0.0, 0.0, -np.inf
                    continue
                vg = v[:keys, h // hpr]
                s = (vg @ q_abs[r0 + i, h, :d_h] + k[:keys] @ q_abs[r0 + i, h, d_h:]) * np.log(2.0)
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                out[r0 + i, h], mag[r0 + i, h] = p @ vg / z, p @ np.abs(vg) / z
                lse[r0 + i, h] = m + np.log(z)
    return out, lse, mag


def verify_draft(vocab, tokens, q_start, target, draft, u_accept, u_sample):
    """(out_tokens, n_accepted, kept - seq_len per request): accept, refuse, redraw.
    Rows of no request stay None."""
    out, acc, delta = [None] * len(tokens), [], []
    for b in range(len(q_start) - 1):
        r0, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        if n == 0:
            acc.append(0)
            delta.append(0)
            continue
        a = 0
        while a < n - 1:
            x = int(tokens[r0 + a + 1])
            if not 0 <= x < vocab:
                break
            q = float(draft[r0 + a][x]) if draft is not None else 1.0
            if not float(u_accept[r0 + a]) * q < float(target[r0 + a][x]):
                break
            a += 1
        p = np.asarray(target[r0 + a][:vocab], dtype=np.float64)
        w = p.copy()
        if a < n - 1:
            x = int(tokens[r0 + a + 1])
            if draft is not None:
                w = p - np.asarray(draft[r0 + a][:vocab], dtype=np.float64)
            elif 0 <= x < vocab:
                w[x] = 0.0
        w = np.where(w > 0, w, 0.0)
        if w.sum() == 0:
            w = np.where(p > 0, p, 0.0)
        reach = np.cumsum(w)
        if reach[-1] > 0:
            over = np.nonzero((reach > float(u_sample[b]) * reach[-1]) & (w > 0))[0]
            v = int(over[0]) if len(over) else int(np.nonzero(w)[0][-1])
        else:
            v = vocab - 1
        for i in range(a):
            out[r0 + i] = int(tokens[r0 + i + 1])
        out[r0 + a] = v
        for i in range(a + 1, n):
            out[r0 + i] = -1
        acc.append(a)
        delta.append(a - (n - 1))
    return out, acc, delta
