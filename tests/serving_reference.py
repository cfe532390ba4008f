"""The serving step's operators from their definitions, in 64 bits on the CPU (numpy and
torch float64): the oracle of the 4-bit cache's and the sampler's tests."""
import math

import numpy as np
import torch


def quantise(x):
    """(codes, scale float16, zero) of the rows of x (float32 arrays), IEEE FP32 as defined."""
    x = np.asarray(x, dtype=np.float32)
    fine = np.isfinite(x).all(-1, keepdims=True)
    x = np.where(fine, x, np.float32(0))
    lo, hi = np.minimum(x.min(-1, keepdims=True), 0), np.maximum(x.max(-1, keepdims=True), 0)
    scale = np.minimum((hi - lo) / np.float32(15), np.float32(65504)).astype(np.float16)
    s32 = scale.astype(np.float32)
    inv = np.where(s32 > 0, np.float32(1) / np.where(s32 > 0, s32, np.float32(1)), np.float32(0)).astype(np.float32)
    zero = np.clip(np.rint(-lo * inv), 0, 15)
    code = np.clip(np.rint(x * inv) + zero, 0, 15)
    scale = np.where(fine, scale, np.float16(np.nan))
    return code.astype(np.uint8), scale[..., 0], zero[..., 0].astype(np.uint8)


def encode(kc, ks, kz, vc, vs, vz):
    """One (page, head) block: codes [P][D] and scales, zeros [P] of K and V -> uint8 [P/16][16 (D + 6)]."""
    P, D = kc.shape
    out = np.zeros((P // 16, 16 * (D + 6)), np.uint8)
    for t in range(P):
        tile, r = out[t // 16], t % 16
        tile[r * D // 2:(r + 1) * D // 2] = kc[t, 0::2] | kc[t, 1::2] << 4
        h, c, e = r // 8, r % 8 // 2, r % 2
        for d in range(0, D, 2):
            n, w, i = d // (D // 8), d % (D // 8) // 4, d % 4
            word = (((h * 8 + n) * 4 + c) * (D // 32) + w) * 2 + e
            tile[8 * D + 2 * word + i // 2] = vc[t, d] | vc[t, d + 1] << 4
        tile[16 * D + 2 * r:16 * D + 2 * r + 2] = np.frombuffer(np.float16(ks[t]).tobytes(), np.uint8)
        tile[16 * D + 32 + 2 * r:16 * D + 34 + 2 * r] = np.frombuffer(np.float16(vs[t]).tobytes(), np.uint8)
        tile[16 * D + 64 + r] = kz[t]
        tile[16 * D + 80 + r] = vz[t]
    return out


def decode(block, D):
    """The reverse: (kc, ks, kz, vc, vs, vz) of uint8 [P/16][16 (D + 6)], vectorised over tokens."""
    T = block.shape[0]
    k = block[:, :8 * D].reshape(T * 16, D // 2)
    kc = np.stack([k & 15, k >> 4], -1).reshape(T * 16, D)
    v = block[:, 8 * D:16 * D].reshape(T, 2, 8, 4, D // 32, 2, 2)      # tile h n c w e byte
    v = np.stack([v & 15, v >> 4], -1)                                 # .. byte, nibble
    vc = v.transpose(0, 1, 3, 5, 2, 4, 6, 7).reshape(T * 16, D)
    f16 = lambda a: np.ascontiguousarray(a).view(np.float16).reshape(-1)
    ks, vs = f16(block[:, 16 * D:16 * D + 32]), f16(block[:, 16 * D + 32:16 * D + 64])
    return kc, ks, block[:, 16 * D + 64:16 * D + 80].reshape(-1), vc, vs, block[:, 16 * D + 80:].reshape(-1)


def attention(q, cache, table, seq, starts, page_size, scale, window):
    """out, lse, and the two error masses of the tolerance, float64. q float64 [T][H][D]; cache uint8 numpy.

    score_mass[t][h]: the largest sum |q| (c + z) s_k scale over visible keys; value_mass[t][h][D]:
    sum p s_v (c + z) / sum p. An entry of the table outside the cache hides its tokens."""
    T, H, D = q.shape
    pages, kv = cache.shape[:2]
    g = H // kv
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    smass, vmass = np.zeros((T, H)), np.zeros((T, H, D))
    for b in range(len(seq)):
        n, a, e = int(seq[b]), int(starts[b]), int(starts[b + 1])
        need = -(-n // page_size)
        ids = np.asarray(table[b, :need])
        hidden = np.repeat((ids < 0) | (ids >= pages), page_size)[:n]
        for h in range(kv):
            if n == 0:
                continue
            block = cache[np.where((ids < 0) | (ids >= pages), 0, ids), h].reshape(-1, 16 * (D + 6))
            kc, ks, kz, vc, vs, vz = [x[:n].astype(np.float64) for x in decode(block, D)]
            pos = np.arange(n - (e - a), n)[:, None]
            col = np.arange(n)[None]
            see = (col <= pos) & ~hidden[None]
            if window > 0:
                see &= col > pos - window
            key = (kc - kz[:, None]) * ks[:, None]
            val = (vc - vz[:, None]) * vs[:, None]
            for j in range(h * g, (h + 1) * g):
                x = np.where(see, 0.0, -np.inf)
                with np.errstate(invalid="ignore"):
                    s = q[a:e, j] @ np.where(hidden[:, None], 0.0, key).T * scale
                x = np.where(see, s, -np.inf)
                for i in range(e - a):
                    v = see[i]
                    if not v.any():
                        continue
                    xs = x[i, v]
                    m = xs.max()
                    p = np.exp(xs - m)
                    l = p.sum()
                    out[a + i, j] = p @ val[v] / l
                    lse[a + i, j] = m + math.log(l) if l == l else np.nan
                    smass[a + i, j] = (np.abs(q[a + i, j]) @ ((kc[v] + kz[v, None]) * ks[v, None]).T).max() * scale
                    vmass[a + i, j] = p @ ((vc[v] + vz[v, None]) * vs[v, None]) / l
    return out, lse, smass, vmass


def tables(seq, new, free, table, page_size, taken):
    """(table, slots, positions, starts, taken) from request lengths, one page and token at a time."""
    table = np.array(table)
    cols = table.shape[1]
    slots, positions, starts = [], [], [0]
    for b, (s, a) in enumerate(zip(seq, new)):
        a = max(int(a), 0)
        count = lambda t: min(cols, -(-max(int(t), 0) // page_size))
        old, want = count(s - a), count(s)
        for c in range(old, cols):
            table[b, c] = -1
            if c < want:
                table[b, c] = free[taken] if taken < len(free) else -1
                taken += 1
        for i in range(a):
            pos = int(s) - a + i
            page = table[b, pos // page_size] if pos >= 0 and pos // page_size < cols else -1
            slots.append(int(page) * page_size + pos % page_size if page >= 0 else -1)
            positions.append(pos)
        starts.append(starts[-1] + a)
    return table, slots, positions, starts, taken


def sample_row(x, u, temperature, top_k, top_p, min_p):
    """Float64 description of one row's draw: (order, before, after, kept) where order ranks the tokens and
    before/after is the running kept weight around each token in index order, as shares of the kept weight."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    n = len(x)
    order = np.argsort(-x, kind="stable")
    rank = np.empty(n, int)
    rank[order] = np.arange(n)
    m = x.max()
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        e = np.where(x == m, 1.0, np.exp((x - m) * (1.0 / temperature if temperature > 0 else 1.0)))
    k = 1 if not temperature > 0 else n if top_k <= 0 else min(n, top_k)
    keep = rank < k
    es = np.where(np.arange(n) < k, e[order], 0.0)
    ranked_before = np.empty(n)
    ranked_before[order] = (np.cumsum(es) - es) / es.sum()
    return rank, e, keep, ranked_before
