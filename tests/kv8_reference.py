"""The 8-bit cache, the rotation and the norms from their definitions (numpy and torch on the CPU): the
oracle of their tests. What is stored is computed in FP32 with IEEE operations, as defined; everything else in 64 bits."""
import math

import numpy as np

F = np.float32


def rope_table(rows, rot, base=10000.0):
    angle = np.arange(rows, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(F)


def rotate(x, positions, table, interleaved):
    """x [tokens][heads][D] of any float type, in that type, each product and sum rounded; rows of positions that the table
    does not have are NaN."""
    rot = table.shape[1]
    pos = np.asarray(positions)
    fine = (pos >= 0) & (pos < table.shape[0])
    at = table[np.where(fine, pos, 0)].astype(x.dtype)[:, None]
    cos, sin = at[..., :rot // 2], at[..., rot // 2:]
    i = np.arange(rot // 2)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., first] = x[..., first] * cos - x[..., second] * sin
        y[..., second] = x[..., second] * cos + x[..., first] * sin
    y[~fine] = np.nan
    return y


def decode(tiles, D):
    """(kc, vc) uint8 [tiles][16][D] and (ks, vs) float32 [tiles] of uint8 [tiles][32 D + 16]."""
    n = tiles.shape[0]
    kc = tiles[:, :16 * D].reshape(n, D // 64, 16, 64).transpose(0, 2, 1, 3).reshape(n, 16, D)
    v = tiles[:, 16 * D:32 * D].reshape(n, D // 64, 2, 8, 4, 4, 2, 2)                # p h n c j e i
    vc = v.transpose(0, 2, 4, 6, 1, 3, 5, 7).reshape(n, 16, D)                       # h c e, p n j i
    scales = np.ascontiguousarray(tiles[:, 32 * D:32 * D + 8]).view(F)
    return kc, vc, scales[:, 0].copy(), scales[:, 1].copy()


def encode(kc, vc, ks, vs, unused=None):
    """The reverse, one tile and byte at a time."""
    n, _, D = kc.shape
    out = np.zeros((n, 32 * D + 16), np.uint8) if unused is None else unused.copy()
    for t in range(16):
        for d in range(D):
            p, r = d // 64, d % 64
            out[:, (p * 16 + t) * 64 + r] = kc[:, t, d]
            h, c, e = t // 8, t % 8 // 2, t % 2
            out[:, 16 * D + ((((p * 2 + h) * 8 + r // 8) * 4 + c) * 4 + r % 8 // 2) * 4 + 2 * e + r % 2] = vc[:, t, d]
    out[:, 32 * D:32 * D + 4] = np.ascontiguousarray(ks.astype(F)).view(np.uint8).reshape(n, 4)
    out[:, 32 * D + 4:32 * D + 8] = np.ascontiguousarray(vs.astype(F)).view(np.uint8).reshape(n, 4)
    return out


def store(code, old, rows, off):
    """One head's codes uint8 [16][D] and scale of a tile after a run's rows (float32 [count][D]) at off: (codes, scale)."""
    top = np.abs(rows).max() if np.isfinite(rows).all() else F(np.nan)
    a = F(top) * (F(1) / F(127))
    if a < F(2.0 ** -40):
        a = F(0)
    a = a if np.isnan(a) else min(a, F(2.0 ** 40))
    old = F(0) if off == 0 else F(old)
    scale = F(np.nan) if np.isnan(a) or np.isnan(old) else max(old, a)
    inv = F(1) / scale if scale > 0 else F(0)
    code = code.copy()
    if scale > old:
        less = np.rint((code[:off].astype(F) - F(128)) * (old * inv))
        code[:off] = (np.clip(less, -127, 127) + 128).astype(np.uint8)
    if scale > 0:
        code[off:off + len(rows)] = (np.clip(np.rint(rows * inv), -127, 127) + 128).astype(np.uint8)
    else:
        code[off:off + len(rows)] = 128
    return code, scale


def append(cache, k, v, slots, page_size):
    """The cache uint8 [pages][heads][page_size / 16][bytes] after k and v float32 [tokens][heads][D], run by run."""
    cache = cache.copy()
    pages, heads, _, size = cache.shape
    D = k.shape[2]
    i = 0
    while i < len(slots):
        s, n = int(slots[i]), 1
        if not 0 <= s < pages * page_size:
            i += 1
            continue
        while i + n < len(slots) and int(slots[i + n]) == s + n and (s + n) % 16 != 0 and s + n < pages * page_size:
            n += 1
        tile = cache[s // page_size, :, s % page_size // 16]                       # [heads][bytes], a view
        kc, vc, ks, vs = decode(tile, D)
        for h in range(heads):
            kc[h], ks[h] = store(kc[h], ks[h], k[i:i + n, h], s % 16)
            vc[h], vs[h] = store(vc[h], vs[h], v[i:i + n, h], s % 16)
        tile[:] = encode(kc, vc, ks, vs, tile)
        i += n
    return cache


def attention(q, cache, table, seq, starts, page_size, scale, window):
    """out, lse and masses for tolerances, float64; q float64 [T][H][D].

    score_mass[t][h]: the largest sum |q| (c + 128) s_k |scale| over visible keys (c the bare code 0 .. 255); value_mass:
    sum p s_v (c + 128) / sum p; and abs_mass: sum p |v| / sum p. An entry of the table outside the cache hides its tokens."""
    T, H, D = q.shape
    pages, kv = cache.shape[:2]
    g = H // kv
    out, vmass, amass = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, smass = np.full((T, H), -np.inf), np.zeros((T, H))
    for b in range(len(seq)):
        n, a, e = int(seq[b]), int(starts[b]), int(starts[b + 1])
        if n == 0 or e == a:
            continue
        held = np.full(-(-n // page_size), -1, np.int64)
        held[:min(len(held), table.shape[1])] = table[b, :len(held)]
        hidden = np.repeat((held < 0) | (held >= pages), page_size)[:n]
        for h in range(kv):
            kc, vc, ks, vs = decode(cache[np.where((held < 0) | (held >= pages), 0, held), h].reshape(-1, 32 * D + 16), D)
            kc, vc = (x.reshape(-1, D)[:n].astype(np.float64) for x in (kc, vc))
            ks, vs = (np.where(hidden, 0.0, np.repeat(x.astype(np.float64), 16)[:n])[:, None] for x in (ks, vs))
            key, val = (kc - 128) * ks, (vc - 128) * vs
            pos, col = np.arange(n - (e - a), n)[:, None], np.arange(n)[None]
            see = (col <= pos) & ~hidden[None]
            if window > 0:
                see &= col > pos - window
            for j in range(h * g, (h + 1) * g):
                with np.errstate(invalid="ignore"):
                    s = q[a:e, j] @ key.T * scale
                    mass = np.abs(q[a:e, j]) @ ((kc + 128) * ks).T * abs(scale)
                for i in range(e - a):
                    w = see[i]
                    if not w.any():
                        continue
                    x = s[i, w]
                    m = x.max()
                    p = np.exp(x - m)
                    l = p.sum()
                    out[a + i, j] = p @ val[w] / l
                    lse[a + i, j] = m + math.log(l) if l == l else np.nan
                    smass[a + i, j] = mass[i, w].max()
                    vmass[a + i, j] = p @ ((vc[w] + 128) * vs[w]) / l
                    amass[a + i, j] = p @ np.abs(val[w]) / l
    return out, lse, smass, vmass, amass
