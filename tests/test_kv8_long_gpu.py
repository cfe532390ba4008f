"""Attention over the 8-bit cache at long contexts, by bounds that zeros, a lost part or a part counted twice do not pass
(tests/kv8_bounds.py), over scales of V as far apart as is promised, and by both kernels whatever max_q says."""
import numpy as np
import pytest

from tests import kv8_reference as ref
from tests.kv8_bounds import bounds, by_blocks

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def requests(seq, nq, heads, group, D, page, dtype, seed, v_scale=None):
    """Queries, a cache with levels of V by blocks and NaN scales in every tile without a token, and the batch's arrays."""
    r = np.random.default_rng(seed)
    held = [-(-s // page) for s in seq]
    ids = r.permutation(sum(held) + 2)
    table = np.full((len(seq), max(held) + 1), -1, np.int32)
    cache = r.integers(0, 256, (len(ids), heads, page // 16, 32 * D + 16), dtype=np.uint8)
    cache[..., 32 * D:32 * D + 8] = np.full(2, np.nan, np.float32).view(np.uint8)
    at = 0
    for b, s in enumerate(seq):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        by_blocks(cache, table[b], s, page, D, seed + b)
        for tile in range(-(-s // 16)):
            sc = np.exp(0.3 * r.standard_normal((heads, 2))).astype(np.float32) * np.float32(0.02)
            if v_scale is not None:
                sc[:, 1] = v_scale(b, tile)
            cache[table[b, tile * 16 // page], :, tile * 16 % page // 16, 32 * D:32 * D + 8] = sc.view(np.uint8)
    starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(starts[-1]), heads * group, D)) * 0.5).to(getattr(torch, dtype))
    return q, cache, table, np.array(seq, np.int32), starts


def run(q, cache, table, seq, starts, page, path, window=0, max_q=None):
    from weight_only_int4_02_gb300 import w4a16
    max_q = int(np.diff(starts).max()) if max_q is None else max_q
    before = w4a16.kv8_force_path(path)
    try:
        out, lse = w4a16.kv8_attention(q.cuda(), *(torch.from_numpy(x).cuda() for x in (cache, table, seq, starts)), page, max_q,
                                       window=window, return_lse=True)
    finally:
        w4a16.kv8_force_path(before)
    assert w4a16.check_device_status() == w4a16.OK
    return out, lse


def inside(args, page, got, path, window=0, more=0.0):
    q, cache, table, seq, starts = args
    o, l, smass, vmass, amass = ref.attention(q.double().numpy(), cache, table, seq, starts, page, q.shape[-1] ** -0.5, window)
    either = [bounds(o, l, smass, vmass, amass, int(seq.max()), which, q.dtype == torch.float16) for which in ((path,) if path else (1, 2))]
    out, log = (np.maximum.reduce(x) for x in zip(*either))   # path 0: whichever kernel's
    err = np.abs(got[0].double().cpu().numpy() - o)
    assert (err <= out + more).all(), "worst error over its bound %.3f" % np.max(err / (out + more))
    g = got[1].double().cpu().numpy()
    fine = np.isfinite(l)
    assert np.array_equal(np.isneginf(g), np.isneginf(l)) and (np.abs(g[fine] - l[fine]) <= log[fine]).all()


@pytest.mark.parametrize("seq,nq,heads,group,D,dtype", [
    (20011, 1, 2, 4, 128, "float16"), (100003, 2, 2, 4, 128, "bfloat16"), (131072, 1, 1, 8, 64, "float16"), (50021, 5, 1, 4, 64, "bfloat16"),
    (33000, 3, 1, 8, 128, "float16"), (9001, 1, 3, 1, 128, "float16")])
def test_few_rows_over_a_long_request(seq, nq, heads, group, D, dtype):
    args = requests([seq], [nq], heads, group, D, 64, dtype, 3)
    got = run(*args, 64, 1)
    inside(args, 64, got, 1)
    again = run(*args, 64, 1)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "float16"), (128, "bfloat16")])
def test_few_rows_of_ragged_requests(D, dtype):
    seq = [20011, 17, 5003, 1, 12001, 777]
    args = requests(seq, [2, 1, 1, 1, 2, 2], 2, 4, D, 32, dtype, 4)
    inside(args, 32, run(*args, 32, 1), 1)
    inside(args, 32, run(*args, 32, 1, window=4001), 1, window=4001)


@pytest.mark.parametrize("seq,nq,heads,group,D,dtype", [
    (9001, 130, 1, 4, 128, "bfloat16"), (20011, 40, 1, 2, 64, "float16"), (20011, 33, 2, 1, 128, "float16"), (33000, 70, 1, 1, 64, "bfloat16")])
def test_many_rows_over_a_long_request(seq, nq, heads, group, D, dtype):
    """One request: its cached tokens are split over several CTAs. And two, with the window's edge far from the end."""
    args = requests([seq], [nq], heads, group, D, 64, dtype, 5)
    got = run(*args, 64, 2)
    inside(args, 64, got, 2)
    again = run(*args, 64, 2)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    args = requests([seq, 3001], [nq, 50], heads, group, D, 64, dtype, 6)
    inside(args, 64, run(*args, 64, 2, window=6001), 2, window=6001)


@pytest.mark.parametrize("path,nq", [(1, 6), (2, 160)])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("apart", [10, 20])
def test_scales_of_v_as_far_apart_as_is_promised(path, nq, dtype, apart):
    """Every fifth tile's scale is 2^apart times the others', which are all that some rows see; and the large ones come late as well. In the
    tcgen05 kernel a weight p of a small tile is fed as p s / S times a number from 64 to 128 (S the largest scale), so that binary16's last
    subnormal, rounded by half a step, is 2^-25 / 64 S |c - 128| of p's sum: with weights all nearly one, 127 * 2^(apart - 31) of the
    small scale for each weight over their mean, which is at most e^3 here (scores within 3 of each other)."""
    page, D, seq, small = 32, 128, 900, 0.02 * 2.0 ** -apart
    for large in (lambda t: t % 5 == 4, lambda t: t >= 50):
        args = requests([seq], [nq], 1, 2, D, page, dtype, 7, v_scale=lambda b, t: 0.02 if large(t) else small)
        args = ((args[0].double() * 0.25).to(args[0].dtype),) + args[1:]
        for window in (0, 37):
            got = run(*args, page, path, window)
            inside(args, page, got, path, window, more=np.exp(3) * 127 * 2.0 ** (apart - 31) * small if path == 2 else 0.0)


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("max_q", [0, 1, 8, 800, 8000])
def test_both_kernels_whatever_max_q_says(D, dtype, max_q):
    """850 tokens of eight heads: enough for the tcgen05 kernel where max_q says that a request has many; the stream-K kernel takes them
    all where it says less."""
    args = requests([900, 300, 65, 40, 1], [801, 1, 38, 9, 1], 2, 4, D, 32, dtype, 8)
    inside(args, 32, run(*args, 32, 0, max_q=max_q), 0)


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("seq,nq,heads,group,max_q", [(300, 20, 128, 1, 20), (300, 20, 128, 1, 1000), (300, 1, 8, 300, 1000), (77, 1, 64, 40, 0),
                                                      (77, 1, 64, 40, 1000), (3, 30, 100, 1, 200)])
def test_one_request_of_few_rows_and_many_heads(seq, nq, heads, group, max_q, D, dtype):
    """Rows of a KV head far fewer than max_q says, in batches of one that are the tcgen05 kernel's alone by it; queries before the
    first token among them."""
    r = np.random.default_rng(9)
    args = requests([seq], [nq], heads, group, D, 16, dtype, 9)
    inside(args, 16, run(*args, 16, 0, max_q=max_q), 0)
