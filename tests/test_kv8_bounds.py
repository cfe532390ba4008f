"""The bounds that long contexts are held to, on the CPU: the definition is inside them, and what a kernel could get wrong is not."""
import numpy as np
import pytest

from tests import kv8_reference as ref
from tests.kv8_bounds import bounds, by_blocks, outside


def request(seq, nq, group, D, page, seed):
    r = np.random.default_rng(seed)
    pages = -(-seq // page)
    table = r.permutation(pages).astype(np.int32)[None]
    cache = r.integers(0, 256, (pages, 1, page // 16, 32 * D + 16), dtype=np.uint8)
    scales = np.exp(0.3 * r.standard_normal((pages, 1, page // 16, 2))).astype(np.float32) * np.float32(0.02)
    cache[..., 32 * D:32 * D + 8] = np.ascontiguousarray(scales).view(np.uint8)
    by_blocks(cache, table[0], seq, page, D, seed)
    q = r.standard_normal((nq, group, D)) * 0.5
    return q, cache, table, np.array([seq]), np.array([0, nq])


def test_levels_are_written_where_the_layout_says():
    _, cache, table, _, _ = request(200, 1, 1, 128, 64, 3)
    _, vc, _, _ = ref.decode(cache[table[0, :4], 0].reshape(-1, 32 * 128 + 16), 128)
    v = vc.reshape(-1, 128)[:192].astype(int).reshape(2, 96, 128)
    assert ((np.abs(v - 78) <= 20).all(1) | (np.abs(v - 178) <= 20).all(1)).all() and (np.abs(v - 78) <= 20).all(1).any()


@pytest.mark.parametrize("seq", [3001, 20011, 100003])
@pytest.mark.parametrize("path,half", [(1, True), (1, False), (2, True), (2, False)])
def test_what_is_wrong_is_outside(seq, path, half):
    D, page = 64, 64
    args = request(seq, 2, 2, D, page, 5)
    o, lse, smass, vmass, amass = ref.attention(*args, page, D ** -0.5, 0)
    out, log = bounds(o, lse, smass, vmass, amass, seq, path, half)
    assert outside(np.zeros_like(o), o, out) > 0.5                       # nothing at all
    assert outside(o * 1.01, o, out) > 0.4                               # a sum of weights off by a hundredth
    rounded = o.astype(np.float16).astype(np.float64) if half else (o * (1 + 2.0 ** -9))
    assert outside(rounded, o, out) == 0
    # a part of the keys left out, or counted twice: from the middle, as CTAs would have it
    q, cache, table, _, _ = args
    raw = cache[table[0], 0].reshape(-1, 32 * D + 16)
    kc, vc, ks, vs = ref.decode(raw, D)
    key, val = (((c.astype(np.float64) - 128) * s[:, None, None]).reshape(-1, D)[:seq] for c, s in ((kc, ks), (vc, vs)))
    for share in (57, 114, 228):
        n = max(16, seq // share // 16 * 16)
        at = seq // 2 // 16 * 16
        for times in (0.0, 2.0):
            w = np.ones(seq)
            w[at:at + n] = times
            got, logs = np.zeros_like(o), np.zeros_like(lse)
            for i in range(2):
                for h in range(2):
                    s = key[:seq - 1 + i] @ q[i, h] * D ** -0.5
                    p = w[:len(s)] * np.exp(s - s.max())
                    got[i, h], logs[i, h] = p @ val[:len(s)] / p.sum(), s.max() + np.log(p.sum())
            assert outside(got, o, out) > 0, (share, times)
            assert (np.abs(logs - lse) > log).all(), (share, times)


def test_the_definition_is_inside():
    """In FP32 from end to end, sums one after the other."""
    seq, D, page = 20011, 64, 64
    q, cache, table, n, starts = request(seq, 1, 2, D, page, 6)
    o, lse, smass, vmass, amass = ref.attention(q, cache, table, n, starts, page, D ** -0.5, 0)
    kc, vc, ks, vs = ref.decode(cache[table[0], 0].reshape(-1, 32 * D + 16), D)
    F = np.float32
    key, val = (((c.astype(F) - F(128)) * s[:, None, None]).reshape(-1, D)[:seq] for c, s in ((kc, ks), (vc, vs)))
    for h in range(2):
        s = (key * q[0, h].astype(F)).cumsum(1, dtype=F)[:, -1] * F(D ** -0.5)
        p = np.exp(s - s.max())
        tiles = [(p[t:t + 16, None] * val[t:t + 16]).sum(0, dtype=F) for t in range(0, seq, 16)]
        got = np.cumsum(tiles, 0, dtype=F)[-1] / p.cumsum(dtype=F)[-1]
        for path in (1, 2):
            out, log = bounds(o, lse, smass, vmass, amass, seq, path, True)
            assert outside(got, o[0, h], out[0, h]) == 0
        assert abs(float(s.max() + np.log(p.sum())) - lse[0, h]) <= log[0, h]
