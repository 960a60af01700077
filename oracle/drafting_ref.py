"""Serving with drafts, forks and several position axes in float64 numpy, from
the definitions: rotations by several axes, attention of a tree of drafted
tokens, and the upkeep of a paged cache.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Arrays are float64 or
integers; caches are [pages, Hkv, page_size, d] as in serving_ref.
"""
import math

import numpy as np


def rope_axes(x, positions, table, axes, rot_offset=0, interleaved=False, inverse=False):
    """x [B, H, L, d]: pair i turned by positions[axes[i]] ([A, B, L])."""
    y = np.array(x, dtype=np.float64)
    table = np.asarray(table, dtype=np.float64)
    half = table.shape[1] // 2
    for i in range(half):
        p = np.asarray(positions[axes[i]])
        turn = np.ones(p.shape, dtype=np.complex128)
        known = (p >= 0) & (p < table.shape[0])
        turn[known] = table[p[known], i] + 1j * table[p[known], half + i]
        if inverse:
            turn = turn.conj()
        a = rot_offset + (2 * i if interleaved else i)
        b = a + (1 if interleaved else half)
        z = (y[..., a] + 1j * y[..., b]) * turn[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def tree_keys(parents, n, window_left=-1):
    """For each of the T tokens of a tree in the slots n - T .. n - 1 the sorted
    keys that it sees (none for padding), and its depth."""
    T = len(parents)
    ctx = n - T
    out = []
    for l in range(T):
        path, at = [], l
        while at >= 0:
            if ctx + at < 0 or parents[at] >= at:
                at = -2
                break
            path.append(at)
            at = int(parents[at])
        if at != -1:
            out.append(([], 0))
            continue
        depth = len(path) - 1
        p = ctx + depth
        lo = 0 if window_left < 0 else max(0, p - window_left)
        near = [i for up, i in enumerate(path) if window_left < 0 or up <= window_left]
        out.append(([*range(lo, max(ctx, 0)), *(ctx + i for i in reversed(near))], depth))
    return out


def tree_decode(q, k_cache, v_cache, block_table, seq_lens, parents, scale, softcap=0.0, window_left=-1, k_scale=None,
                v_scale=None):
    """(out, lse, weight, reach) as serving_ref.decode, for a tree of q's tokens."""
    B, Hq, T, _ = q.shape
    Hkv, page, dv = k_cache.shape[1], k_cache.shape[2], v_cache.shape[3]
    out = np.zeros((B, Hq, T, dv))
    weight = np.zeros_like(out)
    lse = np.full((B, Hq, T), -math.inf)
    reach = np.zeros((B, Hq, T))
    G = Hq // Hkv
    for b in range(B):
        for l, (keys, _) in enumerate(tree_keys(parents[b], int(seq_lens[b]), window_left)):
            if not keys:
                continue
            js = np.asarray(keys)
            at = np.asarray(block_table)[b, js // page]
            for g in range(Hkv):
                k = k_cache[at, g, js % page] * (1.0 if k_scale is None else float(k_scale[g]))
                v = v_cache[at, g, js % page] * (1.0 if v_scale is None else float(v_scale[g]))
                x = q[b, g * G:(g + 1) * G, l]
                s = scale * (x @ k.T)
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(1, keepdims=True)
                rows = slice(g * G, (g + 1) * G)
                out[b, rows, l] = (e @ v) / z
                weight[b, rows, l] = (e @ np.abs(v)) / z
                lse[b, rows, l] = (m + np.log(z))[:, 0]
                reach[b, rows, l] = scale * (np.abs(x) @ np.abs(k).T).max(1)
    return out, lse, weight, reach


def compact(cache, block_table, src, start):
    """The cache after each sequence's tokens src[b] have become those at
    start[b], start[b] + 1, ... (a row's list ends at its first negative entry)."""
    old, out, page = np.asarray(cache), np.array(cache), cache.shape[2]
    for b, line in enumerate(src):
        for m, s in enumerate(line):
            if s < 0:
                break
            d = int(start[b]) + m
            out[block_table[b][d // page], :, d % page] = old[block_table[b][s // page], :, s % page]
    return out


def copy(cache, copies):
    """The cache after the page copies (source, destination, rows)."""
    old, out = np.asarray(cache), np.array(cache)
    for a, b, n in copies:
        if a >= 0 and b >= 0 and n > 0:
            out[b, :, :n] = old[a, :, :n]
    return out


def remap(table, parents, keep, room, refs, page):
    """(new_table, refs_out, copies, short) as lists."""
    cols = len(table[0]) if len(table) else None
    pages = len(refs)
    is_page = lambda p: 0 <= p < pages  # noqa: E731
    free = [p for p in range(pages) if refs[p] == 0]
    uses = list(refs)
    for row in table:
        for p in row:
            if is_page(p):
                uses[p] -= 1
    held, users = [], {}  # pages that row i keeps, whether in whole; rows that keep a page
    for i, parent in enumerate(parents):
        n = keep[i] if parent >= 0 else 0
        held.append([(table[parent][j], (j + 1) * page <= n) for j in range(-(-n // page))])
        for p, whole in held[i]:
            if is_page(p):
                users.setdefault(p, []).append((i, whole))
    new, copies, wanted = [], [], 0
    given = iter(free)
    for i, parent in enumerate(parents):
        row, copied = [], [-1, -1, 0]
        for p, whole in held[i]:
            if whole or not is_page(p):
                row.append(p if is_page(p) else -1)
                continue
            alone = uses[p] == 0 and not any(w for _, w in users[p]) and users[p][0][0] == i
            if alone:
                row.append(p)
                continue
            wanted += 1
            to = next(given, -1)
            row.append(to)
            if to >= 0:
                copied = [p, to, keep[i] % page]
        total = -(-max(room[i], keep[i] if parent >= 0 else 0) // page)
        while len(row) < total:
            wanted += 1
            row.append(next(given, -1))
        new.append(row)
        copies.append(copied)
    width = cols if cols is not None else max(map(len, new))
    new = [row + [-1] * (width - len(row)) for row in new]
    out = list(refs)
    for rows, sign in ((table, -1), (new, 1)):
        for row in rows:
            for p in row:
                if is_page(p):
                    out[p] += sign
    return new, out, copies, max(0, wanted - len(free))
