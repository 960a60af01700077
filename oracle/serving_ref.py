"""The serving operators in float64 numpy, from their definitions: rotary
positions, appending to a paged cache, attention over the pages.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Arrays are float64 or
integers; caches are float64 arrays of the values that the device's cache
stands for ([pages, Hkv, page_size, d], for e4m3 before the scale).
"""
import math

import numpy as np

E4M3_MAX = 448.0


def rope(x, positions, table, rot_offset=0, interleaved=False, inverse=False):
    """x [B, H, L, d] turned by positions [B, L]: each pair as a complex
    number times cos + i sin (conjugated for the inverse)."""
    y = np.array(x, dtype=np.float64)
    table = np.asarray(table, dtype=np.float64)
    half = table.shape[1] // 2
    p = np.asarray(positions)
    turn = np.ones(p.shape + (half,), dtype=np.complex128)
    known = (p >= 0) & (p < table.shape[0])
    turn[known] = table[p[known], :half] + 1j * table[p[known], half:]
    if inverse:
        turn = turn.conj()
    for i in range(half):
        a = rot_offset + (2 * i if interleaved else i)
        b = a + (1 if interleaved else half)
        z = (y[..., a] + 1j * y[..., b]) * turn[:, None, :, i]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def e4m3_step(x):
    """The distance between neighbouring e4m3 values around |x| (4 exponent
    bits with bias 7, 3 mantissa bits, smallest normal 2^-6)."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 2.0 ** (np.minimum(e, 8) - 3)


def append(cache, x, block_table, positions, seq_ids=None, scale=None):
    """The cache after the rows x [B, H, L, d] are stored, and a boolean array
    of the rows [pages, page_size] that were written."""
    out = np.array(cache, dtype=np.float64)
    page = out.shape[2]
    written = np.zeros((out.shape[0], page), dtype=bool)
    for b in range(x.shape[0]):
        for l in range(x.shape[2]):
            p = int(positions[b][l])
            if p < 0:
                continue
            at = int(block_table[b if seq_ids is None else int(seq_ids[b][l])][p // page])
            for h in range(x.shape[1]):
                y = x[b, h, l]
                out[at, h, p % page] = y if scale is None else np.clip(y / scale[h], -E4M3_MAX, E4M3_MAX)
            written[at, p % page] = True
    return out, written


def decode(q, k_cache, v_cache, block_table, seq_lens, scale, softcap=0.0, window_left=-1, k_scale=None, v_scale=None):
    """(out, lse, weight, reach) of q [B, Hq, Lq, dqk]: weight = sum_j p_j |v_j|
    and reach = max_j scale sum_d |q_d k_jd| serve the error bounds."""
    B, Hq, Lq, _ = q.shape
    Hkv, page, dv = k_cache.shape[1], k_cache.shape[2], v_cache.shape[3]
    out = np.zeros((B, Hq, Lq, dv))
    weight = np.zeros_like(out)
    lse = np.full((B, Hq, Lq), -math.inf)
    reach = np.zeros((B, Hq, Lq))
    for b in range(B):
        n = int(seq_lens[b])
        for l in range(Lq):
            p = n - Lq + l
            lo = 0 if window_left < 0 else max(0, p - window_left)
            js = np.arange(lo, p + 1)
            if p < 0 or js.size == 0:
                continue
            at = np.asarray(block_table)[b, js // page]
            for h in range(Hq):
                g = h // (Hq // Hkv)
                k = k_cache[at, g, js % page] * (1.0 if k_scale is None else float(k_scale[g]))
                v = v_cache[at, g, js % page] * (1.0 if v_scale is None else float(v_scale[g]))
                s = scale * (k @ q[b, h, l])
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                m = s.max()
                e = np.exp(s - m)
                z = e.sum()
                out[b, h, l] = (e @ v) / z
                weight[b, h, l] = (e @ np.abs(v)) / z
                lse[b, h, l] = m + math.log(z)
                reach[b, h, l] = scale * (np.abs(k) @ np.abs(q[b, h, l])).max()
    return out, lse, weight, reach
