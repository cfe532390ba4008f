"""The 8-bit key-value cache on the GPU against its definition: append (with the rotation) and read byte for byte, attention by both
kernels in 64 bits, at the lengths, head layouts, strides and masks where they can go wrong.

Tolerance of attention. Scores: FP32 sums of D products of q and bare codes in MMAs that round towards zero (eight of 16 products, at most
2^-23 each of the running sum, which the mass sum |q| (c + 128) s_k bounds): 16 * 2^-24 of it. A probability's relative error is its
score's twice over (its own and the maximum's) and the exponential's, 2^-21. A tile's sum of p (c - 128) starts at -128 sum(p): three MMAs of
sums below the mass sum p (c + 128) s_v, and P in two binary16 parts, 2^-22: within 2^-21 twice over; running sums over the keys add
2^-24 a tile. Outputs are rounded by half a step. The tcgen05 kernel rounds probabilities times V's scale to binary16
once for bfloat16 outputs: 2^-11 of sum p |v|."""
import numpy as np
import pytest

from tests import kv8_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"float16": torch.float16, "bfloat16": torch.bfloat16}
NAN = np.frombuffer(np.float32(np.nan).tobytes(), np.uint8)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


# ---------------------------------------------------------------- append and read
def same_cache(got, want, D):
    """Byte for byte, but for which NaN a scale is."""
    got = got.cpu().numpy()
    scales = lambda a: np.ascontiguousarray(a[..., 32 * D:32 * D + 8]).view(np.float32)
    nan = np.isnan(scales(want))
    assert np.array_equal(np.isnan(scales(got)), nan)
    same = got == want
    same[..., 32 * D:32 * D + 8] |= np.repeat(nan, 4, -1)
    assert same.all(), np.argwhere(~same)[:5]


def check_read(cache, slots, page, D):
    from weight_only_int4_02_gb300 import w4a16
    a = cache.cpu().numpy()
    fine = (slots >= 0) & (slots < a.shape[0] * page)
    s = np.where(fine, slots, 0)
    tiles = a[s // page, :, s % page // 16]                                   # [tokens][heads][bytes]
    kc, vc, ks, vs = ref.decode(tiles.reshape(-1, tiles.shape[-1]), D)
    row = np.repeat(s % 16, a.shape[1])
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        for got, c, sc in zip(w4a16.kv8_read(cache, cuda(slots), page, dtype=dtype), (kc, vc), (ks, vs)):
            want = (c[np.arange(len(row)), row].astype(np.float32) - np.float32(128)) * sc[:, None]
            want = np.where(fine[:, None, None], want.reshape(len(slots), -1, D), np.float32(0))
            want = torch.from_numpy(want).to(dtype)
            assert torch.equal(torch.nan_to_num(got.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
            assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))


def rows(tokens, heads, D, seed, dtype):
    r = np.random.default_rng(seed)
    x = r.standard_normal((tokens, heads, D)) * np.exp(r.standard_normal((tokens, heads, 1)))
    return torch.from_numpy(x).to(dtype)


def slots_of(requests, page, pages, seed):
    """Slots of requests (tokens before, new ones), each from its own pages in any order."""
    ids = np.random.default_rng(seed).permutation(pages)
    out, at = [], 0
    for before, new in requests:
        pos = np.arange(before, before + new)
        out.append(ids[at + pos // page] * page + pos % page)
        at += -(-(before + new) // page)
    assert at <= pages
    return np.concatenate(out).astype(np.int64)


LISTS = {"one": [(0, 1)], "decode": [(i, 1) for i in range(1, 18)], "chunks": [(0, 40), (5, 11), (15, 1), (15, 2), (31, 66), (7, 3)],
         "tiles": [(0, 16), (16, 16), (0, 160)], "long": [(9, 1500), (0, 33)]}


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "float16"), (64, "bfloat16"), (128, "bfloat16")])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 32), (8, 256)])
@pytest.mark.parametrize("which", list(LISTS))
def test_append_and_read(D, dtype, heads, page, which):
    from weight_only_int4_02_gb300 import w4a16
    requests = LISTS[which]
    tokens = sum(n for _, n in requests)
    pages = sum(-(-(b + n) // page) for b, n in requests) + 2
    slots = slots_of(requests, page, pages, tokens)
    k, v = rows(tokens, heads, D, 1, DT[dtype]), rows(tokens, heads, D, 2, DT[dtype])
    r = np.random.default_rng(tokens)
    before = r.integers(0, 256, (pages, heads, page // 16, 32 * D + 16), dtype=np.uint8)
    old = 0.02 * np.exp(r.standard_normal((pages, heads, page // 16, 2))).astype(np.float32)
    before[..., 32 * D:32 * D + 8] = np.ascontiguousarray(old).view(np.uint8)
    wide = torch.zeros((tokens, 2 * heads + 1, D), dtype=DT[dtype])   # slices of a wider tensor
    wide[:, :heads], wide[:, heads + 1:] = k, v
    wide = wide.cuda()
    cache = cuda(before)
    w4a16.kv8_append(wide[:, :heads], wide[:, heads + 1:], cuda(slots), cache, page)
    same_cache(cache, ref.append(before, k.float().numpy(), v.float().numpy(), slots, page), D)
    check_read(cache, slots, page, D)


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 24), (128, 128), (128, 16), (128, 104)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("which", ["decode", "chunks", "long"])
def test_append_turns_the_keys(D, rot, interleaved, dtype, which):
    from weight_only_int4_02_gb300 import w4a16
    requests, heads, page = LISTS[which], 3, 32
    tokens = sum(n for _, n in requests)
    pages = sum(-(-(b + n) // page) for b, n in requests) + 1
    slots = slots_of(requests, page, pages, 3)
    pos = np.concatenate([np.arange(b, b + n) for b, n in requests]).astype(np.int32) * 3
    table = ref.rope_table(int(pos.max()) + 1, rot)
    k, v = rows(tokens, heads, D, 1, DT[dtype]), rows(tokens, heads, D, 2, DT[dtype])
    cache = w4a16.kv8_cache(pages, heads, D, page)
    before = cache.cpu().numpy()
    w4a16.kv8_append(k.cuda(), v.cuda(), cuda(slots), cache, page, positions=cuda(pos), rope=cuda(table), interleaved=interleaved)
    turned = ref.rotate(k.float().numpy(), pos, table, interleaved)
    same_cache(cache, ref.append(before, turned, v.float().numpy(), slots, page), D)


@pytest.mark.parametrize("D", [64, 128])
def test_a_request_token_by_token_and_again(D):
    """Scales grow and codes are rounded again, call by call; drafts that were not accepted are written again; a tile
    begun again forgets what it held."""
    from weight_only_int4_02_gb300 import w4a16
    heads, page = 2, 16
    cache = w4a16.kv8_cache(3, heads, D, page)
    want = cache.cpu().numpy()
    k, v = rows(60, heads, D, 5, torch.bfloat16), rows(60, heads, D, 6, torch.bfloat16)
    at = 0
    for first, count in [(0, 3)] + [(i, 1) for i in range(3, 20)] + [(20, 5), (21, 4), (25, 9), (0, 1), (1, 2), (16, 20)]:
        x, y = (t[at % 40:at % 40 + count] for t in (k, v))
        slots = np.arange(first, first + count)
        w4a16.kv8_append(x.cuda(), y.cuda(), cuda(slots), cache, page)
        want = ref.append(want, x.float().numpy(), y.float().numpy(), slots, page)
        same_cache(cache, want, D)
        at += count


def test_slots_outside_the_cache_are_skipped_and_read_zero():
    from weight_only_int4_02_gb300 import w4a16
    D, page = 64, 16
    cache = w4a16.kv8_cache(3, 2, D, page)
    k = rows(9, 2, D, 1, torch.float16)
    slots = np.array([-1, 0, 1, 47, 48, 49, 1 << 40, -16, 16])   # 47 -> 48 leaves the cache
    w4a16.kv8_append(k.cuda(), k.cuda(), cuda(slots), cache, page)
    want = ref.append(np.zeros((3, 2, 1, 32 * D + 16), np.uint8), k.float().numpy(), k.float().numpy(), slots, page)
    same_cache(cache, want, D)
    check_read(cache, slots, page, D)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_extreme_rows(dtype):
    """Zeros, subnormals, magnitudes past the largest scale, infinities and NaN: by tile and head."""
    from weight_only_int4_02_gb300 import w4a16
    D, page = 128, 16
    x = rows(16 * 8, 2, D, 3, torch.float32)
    x[0:16] = 0.0
    x[16:32] *= 2.0 ** -20
    x[32:48] *= 2.0 ** -36       # bfloat16: the scale is below 2^-40; binary16: all zero
    x[48:64] *= 2.0 ** 60 if dtype == "bfloat16" else 2.0 ** 12
    x[64 + 3, 0, 7] = np.inf
    x[80 + 9, 1, 100] = np.nan
    x[96:112] = -np.abs(x[96:112])
    x = x.clamp(-6e4, 6e4).where(torch.isinf(x), x.clamp(-6e4, 6e4)) if dtype == "float16" else x
    x = x.to(DT[dtype])
    x[64 + 3, 0, 7] = np.inf
    cache = w4a16.kv8_cache(8, 2, D, page)
    slots = np.arange(128)
    w4a16.kv8_append(x.cuda(), (-x).cuda(), cuda(slots), cache, page)
    want = ref.append(np.zeros((8, 2, 1, 32 * D + 16), np.uint8), x.float().numpy(), (-x).float().numpy(), slots, page)
    same_cache(cache, want, D)
    scales = np.ascontiguousarray(want[..., 32 * D:32 * D + 8]).view(np.float32)
    assert np.isnan(scales[4, 0]).all() and not np.isnan(scales[4, 1]).any() and np.isnan(scales[5, 1]).all() and (scales[0] == 0).all()
    # the next run of a poisoned tile leaves it poisoned; begun again it is clean
    y = rows(3, 2, D, 4, DT[dtype])
    w4a16.kv8_append(y.cuda(), y.cuda(), cuda(np.array([64 + 5, 64 + 6, 80])), cache, page)
    want = ref.append(want, y.float().numpy(), y.float().numpy(), [64 + 5, 64 + 6, 80], page)
    same_cache(cache, want, D)


def test_positions_that_the_table_does_not_have_show():
    from weight_only_int4_02_gb300 import w4a16
    D, page = 64, 16
    k = rows(4, 2, D, 1, torch.float16).cuda()
    for bad in (-1, 10, 1 << 30):
        cache = w4a16.kv8_cache(2, 2, D, page)
        pos = torch.tensor([0, 9, bad, 3], dtype=torch.int32, device="cuda")
        w4a16.kv8_append(k, k, torch.tensor([0, 1, 16, -1], device="cuda"), cache, page, positions=pos, rope=w4a16.rope_table(10, D))
        rk, rv = w4a16.kv8_read(cache, torch.tensor([0, 1, 16], device="cuda"), page)
        assert torch.isnan(rk[2]).all() and not torch.isnan(rk[:2]).any() and not torch.isnan(rv).any()


def test_many_tokens_take_the_wide_windows():
    """Batches past the sizes at which a warp looks at more of the list, decodes and chunks mixed; 3001 single tokens too."""
    from weight_only_int4_02_gb300 import w4a16
    r = np.random.default_rng(0)
    D, heads, page = 64, 1, 16
    for requests in ([(int(b), 1) for b in r.integers(0, 32, 3001)],
                     [(int(b), int(n)) for b, n in zip(r.integers(0, 40, 150), r.integers(1, 40, 150))]):
        tokens = sum(n for _, n in requests)
        pages = sum(-(-(b + n) // page) for b, n in requests) + 1
        slots = slots_of(requests, page, pages, 1)
        k, v = rows(tokens, heads, D, 1, torch.bfloat16), rows(tokens, heads, D, 2, torch.bfloat16)
        before = r.integers(0, 256, (pages, heads, 1, 32 * D + 16), dtype=np.uint8)
        before[..., 32 * D:32 * D + 8] = np.ascontiguousarray(r.random((pages, heads, 1, 2)).astype(np.float32) * 0.04).view(np.uint8)
        cache = cuda(before)
        w4a16.kv8_append(k.cuda(), v.cuda(), cuda(slots), cache, page)
        same_cache(cache, ref.append(before, k.float().numpy(), v.float().numpy(), slots, page), D)


def test_append_on_a_stream_and_captured():
    from weight_only_int4_02_gb300 import w4a16
    D, page = 128, 32
    k, v = (rows(40, 2, D, s, torch.float16).cuda() for s in (1, 2))
    slots, pos, table = torch.arange(40, device="cuda") + 3, torch.arange(40, dtype=torch.int32, device="cuda"), w4a16.rope_table(64, D)
    want = w4a16.kv8_cache(2, 2, D, page)
    w4a16.kv8_append(k, v, slots, want, page, positions=pos, rope=table)
    other, third = w4a16.kv8_cache(2, 2, D, page), w4a16.kv8_cache(2, 2, D, page)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    w4a16.kv8_append(k, v, slots, other, page, positions=pos, rope=table, stream=s)
    rk, rv = w4a16.kv8_read(other, slots, page, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4a16.kv8_append(k, v, slots, third, page, positions=pos, rope=table)
    third.zero_()
    g.replay()
    assert torch.equal(other, want) and torch.equal(third, want) and torch.equal(rk, w4a16.kv8_read(want, slots, page)[0])


def test_offsets_past_32_bits():
    from weight_only_int4_02_gb300 import w4a16
    page, D, heads = 256, 128, 2
    pages = (5 << 30) // w4a16.kv8_page_bytes(heads, D, page)
    cache = torch.empty((pages, heads, page // 16, 32 * D + 16), dtype=torch.uint8, device="cuda")
    k, v = (torch.randn(300, heads, D, device="cuda", dtype=torch.float16) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    slots = torch.cat([torch.arange(256) + (pages - 1) * page, torch.arange(44) + (pages - 2) * page]).cuda()
    w4a16.kv8_append(k, v, slots, cache, page)
    small = w4a16.kv8_cache(2, heads, D, page)
    w4a16.kv8_append(k, v, torch.arange(300, device="cuda"), small, page)
    assert torch.equal(cache[pages - 1], small[0])
    seq, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([300], [0, 1]))
    near = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    for path in (1, 2):
        q = torch.randn(1, 128, D, device="cuda", dtype=torch.float16)
        before = w4a16.kv8_force_path(path)
        try:
            assert torch.equal(w4a16.kv8_attention(q, cache, table, seq, starts, page, 1), w4a16.kv8_attention(q, small, near, seq, starts, page, 1))
        finally:
            w4a16.kv8_force_path(before)


# ---------------------------------------------------------------- attention
def batch_of(seq, nq, heads, group, D, page, dtype, seed, spread=0.3):
    """A cache filled through its definition, with NaN scales in every tile without a token."""
    r = np.random.default_rng(seed)
    held = [-(-s // page) for s in seq]
    pages = sum(held) + 2
    ids = r.permutation(pages)
    cols = max(held + [1]) + 1
    table = np.full((len(seq), cols), -1, np.int32)
    cache = r.integers(0, 256, (pages, heads, page // 16, 32 * D + 16), dtype=np.uint8)
    cache[..., 32 * D:32 * D + 8] = np.tile(NAN, 2)
    at = 0
    for b, s in enumerate(seq):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        for j in range(held[b]):
            tiles = -(-min(page, s - j * page) // 16)
            sc = np.exp(spread * r.standard_normal((heads, tiles, 2))).astype(np.float32) * np.float32(0.02)
            cache[table[b, j], :, :tiles, 32 * D:32 * D + 8] = np.ascontiguousarray(sc).view(np.uint8)
    starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(starts[-1]), heads * group, D)) * 0.5).to(DT[dtype])
    return q, cache, table, np.array(seq, np.int32), starts


def check(q, cache, table, seq, starts, page, window, out, lse, scale=None, path=1):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    o, l, smass, vmass, amass = ref.attention(q.double().numpy(), cache, table, seq, starts, page, scale, window)
    es = 16 * 2.0 ** -24 * smass
    n = 2.0 ** -24 * (np.max(seq, initial=0) + 64)
    ep = (2 * es + 2.0 ** -21)[..., None] + n
    u = 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -8
    bound = u * np.abs(o) * 1.01 + vmass * ep * 2 + 2.0 ** -24
    if path != 1 and q.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -11 * amass
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(o))
    err = np.where(np.isnan(o), 0.0, np.abs(got - o))
    assert (err <= np.where(np.isnan(o), 1.0, bound)).all(), "worst error over bound %.3f" % np.nanmax(err / bound)
    if lse is not None:
        g = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(g), np.isneginf(l)) and np.array_equal(np.isnan(g), np.isnan(l))
        f = np.isfinite(l)
        assert (np.abs(g[f] - l[f]) <= (2 * es + 2.0 ** -21 + n + 2.0 ** -23 * np.abs(np.where(f, l, 0)))[f]).all()


def run(q, cache, table, seq, starts, page, window=0, path=0, **kw):
    from weight_only_int4_02_gb300 import w4a16
    max_q = int(np.max(np.diff(starts), initial=0))
    before = w4a16.kv8_force_path(path)
    try:
        r = w4a16.kv8_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), page, max_q, window=window,
                                return_lse=True, **kw)
    finally:
        w4a16.kv8_force_path(before)
    assert w4a16.check_device_status() == w4a16.OK
    return r


def run_and_check(args, page, window=0, path=0, **kw):
    r = run(*args, page, window, path, **kw)
    check(*args, page, window, *r, path=path, **kw)
    return r


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "float16"), (64, "bfloat16"), (128, "bfloat16")])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (2, 8), (1, 16), (1, 20)])
def test_decode_lengths(D, dtype, heads, group):
    seq = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 257, 700]
    for page, window in ((16, 0), (64, 0), (32, 40)):
        run_and_check(batch_of(seq, [1] * len(seq), heads, group, D, page, dtype, heads * 10 + group), page, window, 1)


@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
@pytest.mark.parametrize("heads,group,nq", [(2, 1, 5), (2, 4, 2), (1, 4, 4), (3, 2, 9), (1, 7, 33), (2, 1, 130), (1, 8, 70)])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_several_queries(D, dtype, heads, group, nq, window):
    seq = [nq, 0, 333, nq + 1, 200 + nq, 3]
    lens = [nq, 1, nq, max(1, nq - 3), 0, min(nq, 3)]
    args = batch_of(seq, lens, heads, group, D, 32, dtype, nq)
    for path in (1, 2):
        run_and_check(args, 32, window, path)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("group,nq", [(4, 4), (3, 5), (8, 4), (4, 6)])
@pytest.mark.parametrize("window", [0, 50])
def test_batches_of_several_queries(D, dtype, group, nq, window):
    """Enough rows that segments of 16 are taken where they pay."""
    r = np.random.default_rng(group * nq)
    lens = r.integers(0, nq + 1, 96)
    lens[:3] = nq
    seq = lens + r.integers(0, 150, 96) * (r.random(96) < 0.9)
    seq[1], seq[2] = 777, max(0, nq - 2)
    args = batch_of([int(x) for x in seq], [int(x) for x in lens], 2, group, D, 16, dtype, nq)
    run_and_check(args, 16, window, 1)


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (64, "bfloat16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("heads,group,lens,seq", [
    (1, 4, [150, 33], [700, 33]), (2, 1, [300, 1, 40], [300, 900, 1000]), (1, 8, [64], [128]), (1, 8, [65], [129]), (1, 3, [100], [383]),
    (2, 4, [40], [3000]), (1, 3, [150, 30], [2500, 1150])])
@pytest.mark.parametrize("window", [0, 129])
def test_prompt_chunks(D, dtype, heads, group, lens, seq, window):
    args = batch_of(seq, lens, heads, group, D, 32, dtype, sum(lens) + D)
    out, lse = run_and_check(args, 32, window, 2)
    again, lse_again = run(*args, 32, window, 2)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_page_sizes_and_a_small_window(page, path):
    run_and_check(batch_of([600, 90], [200, 90], 1, 2, 128, page, "bfloat16", page), page, 7, path)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("D", [64, 128])
def test_more_queries_than_tokens_leave_rows_empty(D, path):
    args = batch_of([3, 40], [90, 33], 2, 2, D, 16, "float16", 5)
    out, lse = run_and_check(args, 16, 0, path)
    assert (out[:87] == 0).all() and torch.isneginf(lse[:87]).all()


@pytest.mark.parametrize("path", [0, 1, 2])
def test_every_path_serves_a_batch_of_prompts_and_decodes(path):
    run_and_check(batch_of([940, 300, 65, 0], [900, 1, 38, 1], 2, 4, 128, 64, "bfloat16", 3), 64, 0, path)


@pytest.mark.parametrize("seq,nq,dtype", [(20011, 1, "float16"), (100003, 2, "bfloat16")])
def test_one_long_request_is_split_over_the_gpu(seq, nq, dtype):
    args = batch_of([seq], [nq], 2, 4, 128, 64, dtype, 3)
    out, _ = run_and_check(args, 64)
    assert torch.equal(out, run(*args, 64)[0])


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_scales_of_many_sizes_and_rising(path, dtype):
    run_and_check(batch_of([900, 131], [40, 35], 1, 2, 128, 16, dtype, 9, spread=1.5), 16, 0, path)
    args = batch_of([900], [60], 1, 2, 128, 16, dtype, 5, spread=0.0)
    q, cache, table, seq, starts = args
    for t in range(0, 900, 16):
        rise = np.array([0.001 * 2.0 ** (t / 150), 0.001 * 2.0 ** (t / 60)], np.float32)
        cache[table[0, t // 16], 0, 0, 32 * 128:32 * 128 + 8] = rise.view(np.uint8)
    run_and_check(args, 16, 0, path)


def test_values_of_any_size_for_few_rows():
    """The stream-K kernel multiplies each tile's sums by V's scale: from 2^-40 to 2^40 none loses another's bits to binary16."""
    q, cache, table, seq, starts = batch_of([600], [3], 1, 2, 128, 16, "bfloat16", 5, spread=0.0)
    for t in range(0, 600, 16):
        v = np.array([0.02, 2.0 ** (-40 if t < 304 else 2)], np.float32)
        cache[table[0, t // 16], 0, 0, 32 * 128:32 * 128 + 8] = v.view(np.uint8)
    table[0, 19:] = -1     # what is left, tokens below 304, has the smallest scales
    out, _ = run(q, cache, table, seq, starts, 16, 0, 1)
    o, _, smass, vmass, _ = ref.attention(q.double().numpy(), cache, table, seq, starts, 16, 128 ** -0.5, 0)
    err = np.abs(out.double().cpu().numpy() - o)
    assert np.abs(o).max() < 2.0 ** -33
    assert (err <= 2.0 ** -8 * 1.01 * np.abs(o) + vmass * 2 * (32 * 2.0 ** -24 * smass[..., None] + 2.0 ** -21 + 2.0 ** -14)).all()


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_other_softmax_scales(scale, path):
    run_and_check(batch_of([300], [80], 1, 2, 64, 16, "float16", 9), 16, 0, path, scale=scale)


def test_large_and_small_queries():
    q, cache, table, seq, starts = batch_of([100, 77, 30], [1, 1, 1], 1, 8, 128, 16, "bfloat16", 6)
    q[0] *= 60.0
    q[1] *= 1e-20
    q[2] = 0
    run_and_check((q, cache, table, seq, starts), 16)


@pytest.mark.parametrize("path,nq", [(1, 2), (1, 20), (2, 50)])
def test_missing_pages_hide_their_tokens(path, nq):
    q, cache, table, seq, starts = batch_of([200, 100], [nq, nq], 2, 2, 64, 16, "float16", 4)
    table[0, 3], table[0, 7], table[1, 0] = -1, cache.shape[0] + 5, -7
    run_and_check((q, cache, table, seq, starts), 16, 0, path)
    table[:] = -1      # every row of every request empty
    out, lse = run(q, cache, table, seq, starts, 16, 0, path)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("path,nq", [(1, 3), (1, 20), (2, 60)])
@pytest.mark.parametrize("which", [0, 1])
def test_a_poisoned_tile_shows_where_it_is_seen_and_nowhere_else(path, nq, which):
    """The tile of tokens 48 to 63 of 60: queries at positions from 48 on see some of it."""
    D = 128
    q, cache, table, seq, starts = batch_of([60, 50], [nq, 1], 1, 4, D, 16, "bfloat16", 4)
    cache[table[0, 3], 0, 0, 32 * D + 4 * which:32 * D + 4 * which + 4] = NAN
    out, lse = run(q, cache, table, seq, starts, 16, 0, path)
    check(q, cache, table, seq, starts, 16, 0, out, lse if which == 0 else None, path=path)
    first = max(0, 48 - (60 - nq))     # the first query that sees token 48
    assert torch.isnan(out[first:nq]).all() and not torch.isnan(out[:first]).any() and not torch.isnan(out[nq:]).any()
    assert which == 0 or not torch.isnan(lse).any()
    # past a window that leaves it out, nobody sees it
    q, cache, table, seq, starts = batch_of([400], [nq], 1, 4, D, 16, "bfloat16", 4)
    cache[table[0, 3], 0, 0, 32 * D + 4 * which:32 * D + 4 * which + 4] = NAN
    out, _ = run(q, cache, table, seq, starts, 16, 400 - nq - 63, path)
    assert not torch.isnan(out).any()


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
def test_the_largest_window_hides_nothing(path, D, dtype):
    args = batch_of([3, 40, 130, 0, 700], [9, 60, 1, 3, 50], 2, 4, D, 16, dtype, 5)
    out, lse = run_and_check(args, 16, 2 ** 31 - 1, path)
    want, want_lse = run(*args, 16, 0, path)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("window", [0, 20, 300])
def test_requests_longer_than_their_table(path, window):
    q, cache, table, seq, starts = batch_of([480, 512, 100, 400], [70, 1, 40, 33], 2, 4, 64, 16, "float16", 7)
    seq = seq + np.array([60, 20, 0, 900], np.int32)
    run_and_check((q, cache, table[:, :30], seq, starts), 16, window, path)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("batch,nq", [(1000, 2), (70, 40)])
def test_batches_of_many_requests(path, batch, nq):
    r = np.random.default_rng(batch)
    lens = r.integers(0, nq + 1, batch)
    seq = (lens + r.integers(0, 60, batch)) * (r.random(batch) < 0.9)
    run_and_check(batch_of([int(x) for x in seq], [int(x) for x in lens], 1, 4, 64, 16, "float16", batch), 16, 0, path)


@pytest.mark.parametrize("path,nq", [(1, 2), (2, 70)])
def test_strided_views_streams_workspaces_and_graphs(path, nq):
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([90, 700, 73], [nq, nq, 1], 2, 4, 128, 32, "float16", 8)
    want, want_lse = run(q, cache, table, seq, starts, 32, 0, path)
    T, H, D = q.shape
    wide = torch.zeros((T + 5, H + 4, D + 8), dtype=q.dtype)      # rows behind the last request
    wide[:T, 2:2 + H, :D] = q
    view = wide.cuda()[:, 2:2 + H, :D]
    out = torch.full((T + 5, H + 1, D + 16), 9.0, dtype=q.dtype, device="cuda")
    wide_table = cuda(np.concatenate([table, np.full_like(table, 1 << 30)], 1))[:, :table.shape[1]]
    ws = torch.zeros(w4a16.kv8_workspace_bytes(), dtype=torch.uint8, device="cuda")
    c, sl, st = cuda(cache), cuda(seq), cuda(starts)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    before = w4a16.kv8_force_path(path)
    try:
        got, lse = w4a16.kv8_attention(view, c, wide_table, sl, st, 32, nq, out=out[:, 1:, :D], return_lse=True, workspace=ws,
                                       stream=stream)
        stream.synchronize()
        assert torch.equal(got[:T], want) and torch.equal(lse[:T], want_lse)
        assert (out[:, 0] == 9.0).all() and (out[:, :, D:] == 9.0).all() and (out[T:] == 9.0).all()
        # two graphs over one workspace, replayed one after the other on new lengths
        graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
        outs = [torch.zeros_like(want), torch.zeros_like(want)]
        for g, o in zip(graphs, outs):
            with torch.cuda.graph(g):
                w4a16.kv8_attention(view[:T], c, wide_table, sl, st, 32, nq, out=o, workspace=ws)
        for lens in ([40, 500, 2], [88, 699, 70]):
            sl.copy_(cuda(np.array(lens, np.int32)))
            for _ in range(2):
                for g in graphs:
                    g.replay()
            torch.cuda.synchronize()
            assert torch.equal(*outs)
            check(q, cache, table, np.array(lens, np.int32), starts, 32, 0, outs[0], None, path=path)
    finally:
        w4a16.kv8_force_path(before)


def test_max_q_only_chooses_the_kernel():
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([90, 200], [3, 40], 1, 4, 64, 16, "bfloat16", 8)
    for max_q in (0, 1, 4, 1000):
        out = w4a16.kv8_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), 16, max_q)
        check(q, cache, table, seq, starts, 16, 0, out, None)


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("group,nq", [(4, 1), (8, 1), (8, 2)])
def test_long_sums_have_no_bias(D, dtype, group, nq):
    """512 requests over one row of 16384 tokens. An MMA rounds towards zero: a tile's sum starts at -128 sum(p) and gains
    sum p c, so its two or three roundings lose less than 2^-23 each of that mass, either way; the FP32 sums over the tiles are rounded to
    nearest: 3 * 2^-24 of the mass for a mean. Outputs are rounded to nearest, which has no bias: five deviations of their mean."""
    from weight_only_int4_02_gb300 import w4a16
    n, seq, page = 512, 16384, 256
    _, cache, table, _, _ = batch_of([seq], [1], 1, group, D, page, dtype, D + group)
    g = torch.Generator(device="cuda").manual_seed(group)
    q = torch.randn(n * nq, group, D, generator=g, device="cuda").to(getattr(torch, dtype))
    lens = torch.full((n,), seq, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, n * nq + 1, nq, dtype=torch.int32, device="cuda")
    before = w4a16.kv8_force_path(1)
    try:
        out = w4a16.kv8_attention(q, cuda(cache), cuda(table).expand(n, -1), lens, starts, page, nq).double()
    finally:
        w4a16.kv8_force_path(before)
    kc, vc, ks, vs = ref.decode(cache[table[0, :seq // page], 0].reshape(-1, 32 * D + 16), D)
    kc, vc, ks, vs = (torch.from_numpy(x.astype(np.float64)).cuda() for x in (kc, vc, ks, vs))
    key, val = (((c - 128) * s[:, None, None]).reshape(-1, D) for c, s in ((kc, ks), (vc, vs)))
    x = q.double().view(n, nq, group, D) @ key.T * D ** -0.5
    pos = torch.arange(seq - nq, seq, device="cuda")[None, :, None, None]
    p = torch.softmax(x.masked_fill(torch.arange(seq, device="cuda") > pos, -np.inf), -1).view(-1, seq)
    o = (p @ val).view(out.shape)
    mass = float((p @ (255 * vs.repeat_interleave(16))).mean())
    u = 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
    noise = 5 * u * float(o.square().mean().sqrt()) / 3 ** 0.5 / out.numel() ** 0.5
    bias = float((out - o).mean())
    assert abs(bias) <= 3 * 2.0 ** -24 * mass + noise, (bias, mass, noise)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 32, True)])
def test_a_step_from_lengths_to_output(D, rot, interleaved):
    """Tables, norms and rotations, append and attention chained over three steps, drafts taken back among them, against attention in
    64 bits over the cache as the definition fills it."""
    from weight_only_int4_02_gb300 import w4a16
    heads, group, page = 2, 4, 16
    cache = w4a16.kv8_cache(40, heads, D, page)
    want = cache.cpu().numpy()
    rope = w4a16.rope_table(200, rot)
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(40, device="cuda").to(torch.int32)
    w = (1 + 0.1 * torch.randn(D, device="cuda")).to(torch.float16)
    taken, seq = None, np.zeros(3, np.int32)
    for new, keep in (([20, 1, 33], [20, 1, 33]), ([4, 4, 4], [1, 4, 2]), ([1, 3, 2], [1, 3, 2])):
        seq = seq + np.array(new, np.int32)
        T = sum(new)
        qkv = torch.randn(T, heads * (group + 2), D, device="cuda", dtype=torch.float16)
        q, k, v = qkv.split([heads * group, heads, heads], 1)
        sl = cuda(seq)
        slots, positions, starts, taken = w4a16.kv4_tables(sl, cuda(np.array(new, np.int32)), free, table, page, T, taken=taken)
        q, _ = w4a16.qk_norm_rope(q, None, positions, rope, q_weight=w, interleaved=interleaved, q_out=q)
        w4a16.kv8_append(k, v, slots, cache, page, positions=positions, rope=rope, interleaved=interleaved)
        out, lse = w4a16.kv8_attention(q, cache, table, sl, starts, page, max(new), return_lse=True)
        turned = ref.rotate(k.float().cpu().numpy(), positions.cpu().numpy(), rope.cpu().numpy(), interleaved)
        want = ref.append(want, turned, v.float().cpu().numpy(), slots.cpu().numpy(), page)
        same_cache(cache, want, D)
        check(q.cpu(), want, table.cpu().numpy(), seq, starts.cpu().numpy(), page, 0, out, lse)
        # drafts that are not kept: the lengths go back, and the tables' pages with them
        seq = seq - np.array(new, np.int32) + np.array(keep, np.int32)


def test_refusals():
    from weight_only_int4_02_gb300 import w4a16
    from tests.test_binding_refusals_gpu import every_other, ints, refused
    cache = w4a16.kv8_cache(3, 2, 64, 16)
    k = torch.randn(5, 2, 64, device="cuda").to(torch.float16)
    slots, pos, table = torch.arange(5, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda"), w4a16.rope_table(9, 64)
    odd = torch.zeros(5, 2, 68, dtype=torch.float16, device="cuda")
    caches = [("cache", cache.to(torch.int8)), ("cache", cache[:, :, 0]), ("cache", cache.cpu()), ("cache", w4a16.kv4_cache(3, 2, 64, 16)),
              ("cache", cache[..., :-16]), ("cache", cache[..., :-16].contiguous()), ("page_size", 32), ("page_size", None),
              ("slots", slots.int()), ("slots", slots[:, None]), ("slots", every_other(slots))]
    turns = [("positions", None), ("positions", pos.long()), ("positions", pos[:4]), ("positions", pos.cpu()), ("rope", None),
             ("rope", table.half()), ("rope", w4a16.rope_table(9, 72)), ("rope", table[:0]), ("rope", table[:, :20].contiguous())]
    for name in ("k", "v"):
        refused(w4a16.kv8_append, dict(k=k, v=k, slots=slots, cache=cache, page_size=16, positions=pos, rope=table),
                caches + turns + [(name, k.float()), (name, k.bfloat16()), (name, k[:4]), (name, k[:, :1]), (name, k[:1].expand(5, -1, -1)),
                                  (name, k[..., :32]), (name, every_other(k)), (name, odd[..., :64]), (name, k[0]), (name, k.cpu()), (name, None)])
    refused(w4a16.kv8_read, dict(cache=cache, slots=slots, page_size=16, dtype=torch.float32), caches + [("dtype", torch.int8)])
    q = torch.randn(3, 4, 64, device="cuda").to(torch.float16)
    bt, seq, starts = ints(0, 1, 2, -1).view(2, 2), ints(20, 5), ints(0, 2, 3)
    ws = torch.zeros(w4a16.kv8_workspace_bytes() + 256, dtype=torch.uint8, device="cuda")
    refused(w4a16.kv8_attention, dict(q=q, cache=cache, block_table=bt, seq_lens=seq, starts=starts, page_size=16, max_q=2, scale=0.1,
                                      window=0, out=torch.empty_like(q), return_lse=True, workspace=ws),
            [c for c in caches if c[0] != "slots"] + [
                ("q", q.float()), ("q", q[:, :3]), ("q", q[..., :32]), ("q", every_other(q)), ("block_table", bt.long()), ("seq_lens", seq.long()),
                ("starts", ints(0, 2)), ("max_q", -1), ("scale", float("nan")), ("window", -1), ("out", q.bfloat16()), ("workspace", ws[:1024])])


def test_nothing_to_do():
    from weight_only_int4_02_gb300 import w4a16
    cache = w4a16.kv8_cache(2, 2, 64, 16)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    z = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    w4a16.kv8_append(z, z, none, cache, 16, positions=none.int(), rope=w4a16.rope_table(4, 64))
    assert w4a16.kv8_read(cache, none, 16)[0].shape == (0, 2, 64) and not cache.any()
