"""Paged attention in fp64: page bookkeeping, cache write with page summaries,
attention of single rows, block choice and block-sparse attention.

Test infrastructure only (see the package docstring).  Plain loops over
requests, rows and heads, written from the definitions; no numpy broadcasting
across rows, so that a row's result depends on nothing but its own inputs.

Conventions: table [B, W]; caches [n_pages, Hkv, P, D]; row r of request
req[r] sees tokens 0 .. length[r] - 1; query head h reads key/value head
h // (Hq // Hkv).
"""
from __future__ import annotations

import math

import numpy as np


def pages_of(n: int, page: int) -> int:
    return -(-int(n) // page)


def release(lens, done, table, free_list, free_pos, page):
    """Returns (lens, free_list, free_pos) after ended requests' pages went back."""
    lens, ring, (taken, back) = list(map(int, lens)), np.array(free_list), map(int, free_pos)
    for b, d in enumerate(done):
        if not d:
            continue
        for j in range(min(max(pages_of(lens[b], page), 0), table.shape[1])):
            ring[back % len(ring)] = table[b, j]
            back += 1
        lens[b] = 0
    return np.array(lens, np.int32), ring, np.array([taken, back], np.int64)


def plan(lens, add, table, free_list, free_pos, page, rows):
    """Returns the dict of paged_plan, with the new table under "table"."""
    table, ring = np.array(table), np.asarray(free_list)
    B, W = table.shape
    taken, back = map(int, free_pos)
    first = taken
    asked_pages = asked_rows = 0
    out = dict(lens=[], cu=[0], page_cu=[0], slot=[], row_req=[], row_len=[], status=[])
    for b in range(B):
        n, m = int(lens[b]), int(add[b])
        if n < 0 or m < 0:
            st = 8
        elif pages_of(n + m, page) > W:
            st = 2
        else:
            need = pages_of(n + m, page) - pages_of(n, page)
            asked_pages += need
            asked_rows += m
            st = 1 if need and asked_pages > back - first else 4 if m and asked_rows > rows else 0
        if st == 0:
            for j in range(pages_of(n, page), pages_of(n + m, page)):
                table[b, j] = ring[taken % len(ring)]
                taken += 1
            for t in range(n, n + m):
                out["slot"].append(int(table[b, t // page]) * page + t % page)
                out["row_req"].append(b)
                out["row_len"].append(t + 1)
            n += m
        out["lens"].append(n)
        out["status"].append(st)
        out["cu"].append(len(out["slot"]))
        out["page_cu"].append(taken - first)
    spare = rows - len(out["slot"])
    for name, fill in (("slot", -1), ("row_req", -1), ("row_len", 0)):
        out[name] += [fill] * spare
    out = {k: np.array(v, np.int32) for k, v in out.items()}
    out["free_pos"] = np.array([taken, back], np.int64)
    out["table"] = table
    return out


def quantise(x):
    """8-bit codes and the power of two of one vector: the least 2^e (e >= -126)
    with max |x| < 2^(e + 7); elements that are not finite count as 0."""
    x = np.where(np.isfinite(x), np.asarray(x, np.float64), 0.0)
    top = float(np.max(np.abs(x)))
    if top == 0.0:
        return np.zeros(x.shape, np.int8), 1.0
    e = max(math.frexp(top)[1] - 7, -126)
    scale = math.ldexp(1.0, e)
    return np.clip(np.rint(x / scale), -127, 127).astype(np.int8), scale


def write(k, v, slot, k_cache, v_cache, codes=None, scale=None):
    """In place on the given arrays."""
    n_pages, Hkv, P, D = k_cache.shape
    for i, s in enumerate(map(int, slot)):
        if 0 <= s < n_pages * P:
            k_cache[s // P, :, s % P] = k[i]
            v_cache[s // P, :, s % P] = v[i]
    if codes is None:
        return
    for s in map(int, slot):
        if 0 <= s < n_pages * P and s % P == P - 1:
            for h in range(Hkv):
                with np.errstate(invalid="ignore"):
                    mean = k_cache[s // P, h].astype(np.float64).sum(0) / P
                codes[s // P, h], scale[s // P, h] = quantise(mean)


def _attend_keys(q, keys, values, scale):
    """One query over given keys: (o, log-sum, sum of weight |v|, max |x|, max sum |q k| scale)."""
    if len(keys) == 0:
        z = np.zeros(values.shape[1])
        return z, -math.inf, z, 0.0, 0.0
    x = (keys @ q) * scale
    top = x.max()
    w = np.exp(x - top)
    tot = w.sum()
    w = w / tot
    return (w @ values, top + math.log(tot), w @ np.abs(values), float(np.abs(x).max()),
            float((np.abs(keys) @ np.abs(q)).max() * abs(scale)))


def attend(q, k_cache, v_cache, table, length, req=None, scale=None, blocks=None, max_len=None):
    """(o, lse, spread) of every row.  ``blocks`` [R, Hkv, K] restricts a row to
    the listed blocks.  spread holds what an error bound needs: sum of weight
    |v| per element, and per (row, head) n, max |x| and max scale sum |q k|."""
    R, Hq, D = q.shape
    n_pages, Hkv, P, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    o, lse = np.zeros((R, Hq, D)), np.full((R, Hq), -math.inf)
    absv, n, xmax, qk = np.zeros((R, Hq, D)), np.zeros((R, Hq)), np.zeros((R, Hq)), np.zeros((R, Hq))
    B, W = table.shape
    for r in range(R):
        b = r if req is None else int(req[r])
        if not 0 <= b < B or length[r] <= 0:
            continue
        seen = min(int(length[r]), W * P if max_len is None else max_len)
        for h in range(Hkv):
            js = range(pages_of(seen, P)) if blocks is None else blocks[r, h]
            ks, vs = [np.zeros((0, D))], [np.zeros((0, D))]
            for j in map(int, js):
                if not 0 <= j < pages_of(seen, P):
                    continue
                page = int(table[b, j])
                if 0 <= page < n_pages:
                    c = min(P, seen - j * P)
                    ks.append(np.asarray(k_cache[page, h, :c], np.float64))
                    vs.append(np.asarray(v_cache[page, h, :c], np.float64))
            ks, vs = np.concatenate(ks), np.concatenate(vs)
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                o[r, g], lse[r, g], absv[r, g], xmax[r, g], qk[r, g] = _attend_keys(
                    np.asarray(q[r, g], np.float64), ks, vs, scale)
                n[r, g] = len(ks)
    return o, lse, dict(absv=absv, n=n, xmax=xmax, qk=qk)


def select(q, codes, scale, table, length, page, n_blocks, req=None, n_sink=1, n_local=1,
           max_len=None):
    """[R, Hkv, n_blocks] int32: the picked blocks, rising, then -1."""
    R, Hq, D = q.shape
    n_pages, Hkv, _ = codes.shape
    B, W = table.shape
    out = np.full((R, Hkv, n_blocks), -1, np.int32)
    for r in range(R):
        b = r if req is None else int(req[r])
        if not 0 <= b < B or length[r] <= 0:
            continue
        nb = pages_of(min(int(length[r]), W * page if max_len is None else max_len), page)
        for h in range(Hkv):
            qs = [quantise(q[r, g]) for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))]
            score = []
            for j in range(nb):
                p = int(table[b, j])
                best = -math.inf
                if j < n_sink or j >= nb - n_local:
                    best = math.inf
                elif 0 <= p < n_pages and not math.isnan(scale[p, h]):
                    c = codes[p, h].astype(np.int64)
                    best = max(int(q8.astype(np.int64) @ c) * s * float(scale[p, h]) for q8, s in qs)
                score.append(best)
            order = sorted(range(nb), key=lambda j: (-score[j], j))[:n_blocks]
            out[r, h, :len(order)] = sorted(order)
    return out
