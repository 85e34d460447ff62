"""Float64 oracle of the serving calls over a KV cache held in 4 bits.

Plain NumPy, row by row, from the definitions in include/dflash.h; shares no
code with the GPU path.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
# every finite e4m3 value by its code (sign bit clear); code 0x7F is a NaN
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def _nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest of a rising grid, the even index on a tie."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def quantise(x: np.ndarray, exp: np.ndarray):
    """x [..., h, D] float64, exp [h]: (codes uint8 [..., h, D], scale codes [..., h, D/16])."""
    x = np.ldexp(x, -np.asarray(exp, np.int64)[:, None])
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    g = np.where(np.isnan(g), 0.0, g)
    s = _nearest_even(np.abs(g).max(-1) / 6, E4M3)
    f = E4M3[s][..., None]
    mag = _nearest_even(np.abs(g) / np.where(f > 0, f, 1.0), E2M1[:8])
    code = np.where(f > 0, mag + 8 * np.signbit(g), 0).astype(np.uint8)
    return code.reshape(x.shape), s.astype(np.uint8)


def values(code: np.ndarray, scale: np.ndarray, exp: np.ndarray) -> np.ndarray:
    v = E2M1[code].reshape(*code.shape[:-1], code.shape[-1] // 16, 16) * E4M3[scale][..., None]
    return np.ldexp(v.reshape(code.shape), np.asarray(exp, np.int64)[:, None])


def put_row(cell: np.ndarray, r: int, kc, ks, vc, vs):
    """Write one row (codes [D], scale codes [D/16]) into the cell, uint8 [18 D]."""
    d = len(kc)
    for i in range(0, d, 2):
        cell[(i // 32) * 256 + r * 16 + (i % 32) // 2] = kc[i] | kc[i + 1] << 4
        cell[8 * d + (i // 2) * 16 + r] = vc[i] | vc[i + 1] << 4
    for g in range(d // 16):
        cell[16 * d + r * (d // 16) + g] = ks[g]
        cell[17 * d + g * 16 + r] = vs[g]


def get_row(cell: np.ndarray, r: int):
    """(kc, ks, vc, vs) of row r."""
    d = len(cell) // 18
    kc, vc = np.empty(d, np.uint8), np.empty(d, np.uint8)
    for i in range(0, d, 2):
        a = cell[(i // 32) * 256 + r * 16 + (i % 32) // 2]
        b = cell[8 * d + (i // 2) * 16 + r]
        kc[i], kc[i + 1], vc[i], vc[i + 1] = a & 15, a >> 4, b & 15, b >> 4
    ks = cell[16 * d + r * (d // 16):16 * d + (r + 1) * (d // 16)].copy()
    vs = np.array([cell[17 * d + g * 16 + r] for g in range(d // 16)], np.uint8)
    return kc, ks, vc, vs


def norm_rope(x, w, pos, theta, eps):
    """x [N, h, D], w [D] or None, pos [N] (negative: zeros are returned)."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w
    a = np.asarray(pos, np.float64)[:, None] * theta ** (-2.0 * np.arange(d // 2) / d)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    u, v = x[..., :d // 2], x[..., d // 2:]
    y = np.concatenate([u * c - v * s, v * c + u * s], -1)
    return np.where((np.asarray(pos) >= 0)[:, None, None], y, 0.0)


def reserve(seq_len, n_new, table, free_list, free_count, page_size, n_tokens, max_tokens, limit):
    """Returns a dict of what dflash_kv_reserve writes, and the status bits by name."""
    B = len(seq_len)
    table = None if table is None else table.copy()
    start, pos, slot = [0], np.full(n_tokens, -1), np.full(n_tokens, -1)
    new_len, status, count = np.array(seq_len), set(), free_count
    for b in range(B):
        n, first = int(n_new[b]), start[-1]
        start.append(first + max(n, 0))
        L = int(seq_len[b])
        if n < 0 or n > max_tokens or L < 0 or L + n > limit or first + n > n_tokens:
            status.add("capacity")
            continue
        if table is not None and n:
            lack = [p for p in range(L // page_size, (L + n - 1) // page_size + 1)
                    if table[b, p] < 0]
            if len(lack) > count:
                status.add("pool_empty")
                continue
            for p in lack:
                count -= 1
                table[b, p] = free_list[count]
        for i in range(n):
            pos[first + i] = L + i
            slot[first + i] = (b * limit + L + i if table is None else
                               table[b, (L + i) // page_size] * page_size + (L + i) % page_size)
        new_len[b] = L + n
    return {"start": np.array(start), "pos": pos, "slot": slot, "new_len": new_len,
            "table": table, "free_count": count, "status": status}


def attention(q, k, v, n_seen, scale):
    """q [T, Hq, D]; k, v [n, Hkv, D]; row t sees the first n_seen[t] rows.
    Returns (out, mean |v| under the same weights, largest scale sum |q||k|)."""
    T, hq, d = q.shape
    group = hq // k.shape[1]
    out, avg, big = np.zeros((T, hq, d)), np.zeros((T, hq, d)), 0.0
    for t in range(T):
        m = int(n_seen[t])
        if m <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:m, h // group], v[:m, h // group]
            x = kk @ q[t, h] * scale
            p = np.exp(x - x.max())
            p /= p.sum()
            out[t, h], avg[t, h] = p @ vv, p @ np.abs(vv)
            big = max(big, float((np.abs(kk) @ np.abs(q[t, h])).max()) * abs(scale))
    return out, avg, big
