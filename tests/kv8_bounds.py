"""How far attention over the 8-bit cache may be off, for long contexts too: what adds up over the tokens is counted as the kernels add it.

A score is a sum of D products of q and bare codes, in MMAs that round towards zero: 16 * 2^-24 of the mass sum |q| (c + 128) s_k (two
chains of at most four MMAs, 2^-23 each of a chain's share, and three roundings of products and sums). A weight is off by its score's error
and the row's reference's, 2^-21 for the exponential and 2^-22 for its two binary16 parts: that much of sum p |v|, and of the output
through the sum of weights.
The stream-K kernel takes a tile's sum from -128 sum(p), so that its three or four MMAs round sums below the mass sum p (c + 128) s_v: 2^-23 each,
and the share of the 128s as much again: 2^-20. Only a tile's own sum has that mass. What runs on from tile to tile is sum p v: 2^-24 of sum p |v| for
each tile of a warp's run, each warp of a CTA and each CTA of a segment. A quarter of the request's tiles is one warp's at
most, and the more CTAs have a part the fewer are a warp's. A lane's sum of weights has two terms a tile.
The tcgen05 kernel multiplies by codes less 128, and its sums run on in tensor memory, rounded towards zero once for each 16 tokens
and binary16 part of the weights: 2^-23 of sum p |v|. For bfloat16 outputs it feeds one part, 2^-11 of sum p |v|.
Outputs are rounded by half a step."""
import numpy as np

CTAS = 1024     # of a segment, at most


def bounds(o, lse, smass, vmass, amass, seq, path, half):
    """Of outputs and log-sums, as kv8_reference.attention gives the first five; seq: cached tokens of the longest request; half: binary16
    outputs, not bfloat16."""
    tiles = -(-seq // 16)
    es = 16 * 2.0 ** -24 * smass
    ep = (2 * es + 2.0 ** -21 + 2.0 ** -22)[..., None]
    parts = min(tiles, CTAS)
    runs = 2.0 ** -24 * (tiles / 4 + parts + 16)
    sums = 2.0 ** -24 * (tiles / 2 + parts + 32)
    if path == 2:
        runs = 2.0 ** -23 * tiles * (2 if half else 1) + 2.0 ** -24 * 32
        sums = 2.0 ** -24 * (seq / 2 + 32)
    own = 2.0 ** -20 * vmass if path == 1 else 0.0
    out = (2.0 ** -11 if half else 2.0 ** -8) * 1.01 * np.abs(o) + ep * (amass + np.abs(o)) + own + runs * amass + sums * np.abs(o) + 2.0 ** -24
    if path == 2 and not half:
        out = out + 2.0 ** -11 * amass
    return out, 2 * es + 2.0 ** -21 + sums + 2.0 ** -23 * np.abs(np.where(np.isfinite(lse), lse, 0))


def by_blocks(cache, table, seq, page, D, seed):
    """V's codes of a request's row of the table, in place: levels 78 or 178 for d and a block of tokens (a 200th of them, 96 or more),
    one level for about four blocks of five, with a spread of 20. So outputs are large beside their bounds, and no block can be left
    out or counted twice without moving some."""
    r = np.random.default_rng(seed)
    block = max(96, seq // 200 // 16 * 16)
    blocks = -(-seq // block)
    level = np.where((r.random((blocks, D)) < 0.2) == (r.random(D) < 0.5), 78, 178)
    for tile in range(-(-seq // 16)):
        t = np.arange(16) + 16 * tile
        code = level[np.minimum(t // block, blocks - 1)] + r.integers(-20, 21, (16, D))
        v = code.astype(np.uint8).reshape(2, 4, 2, D // 64, 8, 4, 2).transpose(3, 0, 4, 1, 5, 2, 6)   # h c e, p n j i -> p h n c j e i
        cache[table[tile * 16 // page], :, tile * 16 % page // 16, 16 * D:32 * D] = v.reshape(-1)


def outside(got, o, bound):
    """The share of values that are further off than the bound."""
    return float((np.abs(got - o) > bound).mean())
