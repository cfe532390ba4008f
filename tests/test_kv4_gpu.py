"""The 4-bit key-value cache on the GPU against its definition in 64 bits: tables, append,
read and attention, at the lengths, head layouts, strides and masks where they can go wrong."""
import numpy as np
import pytest

from tests import serving_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


# ---------------------------------------------------------------- tables
@pytest.mark.parametrize("batch,page,cols,hi,short", [
    (1, 16, 1, 16, 0), (1, 64, 9, 300, 0), (7, 16, 37, 500, 0), (8, 32, 40, 1000, 0), (9, 16, 30, 600, 5),
    (300, 256, 13, 4000, 0), (1000, 16, 129, 2000, 17), (2500, 32, 6, 200, 0)])
def test_tables(batch, page, cols, hi, short):
    from weight_only_int4_02_gb300 import w4a16
    r = np.random.default_rng(batch + cols)
    seq = r.integers(0, hi + 1, batch).astype(np.int32)
    new = np.where(r.random(batch) < 0.5, 1, r.integers(-1, 90, batch)).astype(np.int32)   # more than seq now and then
    if batch > 4:
        seq[2], new[2] = 0, 0
        seq[3], new[3] = hi, 0
    need = int(sum(max(0, min(cols, -(-int(s) // page)) - min(cols, -(-max(int(s) - max(int(a), 0), 0) // page)))
                   for s, a in zip(seq, new)))
    free = r.permutation(need + 50).astype(np.int32)[:max(0, need + 3 - short)]
    held = r.integers(0, 1 << 27, (batch, cols)).astype(np.int32)      # slots pass 31 bits
    tokens = int(np.maximum(new, 0).sum()) + 5
    want = ref.tables(seq, new, free, held, page, 3)
    table = cuda(held)
    slots, positions, starts, taken = w4a16.kv4_tables(cuda(seq), cuda(new), cuda(free), table, page, tokens,
                                                       taken=torch.full((1,), 3, dtype=torch.int32, device="cuda"))
    assert np.array_equal(table.cpu().numpy(), want[0])
    n = len(want[1])
    assert slots[:n].tolist() == want[1] and (slots[n:] == -1).all()
    assert positions[:n].tolist() == want[2] and (positions[n:] == -1).all()
    assert starts.tolist() == want[3] and taken.item() == want[4]
    # without a count of taken pages: from the first; fewer places than tokens: the first ones
    table = cuda(held)
    few = w4a16.kv4_tables(cuda(seq), cuda(new), cuda(free), table, page, n // 2)
    want = ref.tables(seq, new, free, held, page, 0)
    assert np.array_equal(table.cpu().numpy(), want[0]) and few[0].tolist() == want[1][:n // 2]
    assert few[2].tolist() == want[3] and few[3].item() == want[4]


def test_tables_of_no_requests():
    from weight_only_int4_02_gb300 import w4a16
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    slots, positions, starts, taken = w4a16.kv4_tables(z, z, z, torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 16, 3)
    assert slots.tolist() == [-1] * 3 and starts.tolist() == [0] and taken.item() == 0


# ---------------------------------------------------------------- append and read
def rows(tokens, heads, D, seed, dtype):
    r = np.random.default_rng(seed)
    x = r.standard_normal((tokens, heads, D)) * np.exp(r.standard_normal((1, heads, D)))
    x[0] = 0.0                                       # a row of zeros
    x[1 % tokens] = np.abs(x[1 % tokens])            # one sign only
    x[2 % tokens] = -np.abs(x[2 % tokens])
    x[3 % tokens] *= 2.0 ** -22                      # binary16 subnormals
    if tokens > 6:
        x[4] *= 30000.0 if dtype == torch.float16 else 1e30
        x[5, :, 3], x[6, :, 5] = np.inf, np.nan
    return torch.from_numpy(np.clip(x, -6e4, 6e4) if dtype == torch.float16 and tokens <= 4 else x).to(dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (5, 3, 16), (37, 2, 64), (200, 8, 32), (33, 1, 256)])
def test_append_and_read(D, dtype, tokens, heads, page):
    from weight_only_int4_02_gb300 import w4a16
    pages = -(-tokens // page) + 3
    r = np.random.default_rng(tokens)
    slots = r.permutation(pages * page)[:tokens].astype(np.int64)
    before = r.integers(0, 256, (pages, heads, page // 16, 16 * (D + 6)), dtype=np.uint8)
    k, v = rows(tokens, heads, D, 1, DT[dtype]), rows(tokens, heads, D, 2, DT[dtype])
    wide = torch.zeros((tokens, 2 * heads + 1, D), dtype=DT[dtype])   # slices of a wider tensor
    wide[:, :heads], wide[:, heads + 1:] = k, v
    wide = wide.cuda()
    cache = cuda(before)
    w4a16.kv4_append(wide[:, :heads], wide[:, heads + 1:], cuda(slots), cache, page)
    want = before.copy()
    kc, ks, kz = ref.quantise(k.float().numpy())
    vc, vs, vz = ref.quantise(v.float().numpy())
    for h in range(heads):
        for pg in np.unique(slots // page):
            parts = [np.array(x) for x in ref.decode(before[pg, h], D)]
            for t in np.nonzero(slots // page == pg)[0]:
                o = slots[t] % page
                for part, new in zip(parts, (kc[t, h], ks[t, h], kz[t, h], vc[t, h], vs[t, h], vz[t, h])):
                    part[o] = new
            want[pg, h] = ref.encode(*parts)
    got = cache.cpu().numpy()
    # a poisoned row's scale is a NaN, whichever; everything else byte for byte
    nan_at = lambda a: np.isnan(np.ascontiguousarray(a[..., 16 * D:16 * D + 64]).view(np.float16))
    assert np.array_equal(nan_at(got), nan_at(want))
    same = got == want
    same[..., 16 * D:16 * D + 64] |= np.repeat(nan_at(want), 2, -1)
    assert same.all()
    for out in (torch.float32, torch.float16, torch.bfloat16):
        rk, rv = w4a16.kv4_read(cache, cuda(slots), page, dtype=out)
        for got_x, (c, s, z) in ((rk, (kc, ks, kz)), (rv, (vc, vs, vz))):
            exact = (c.astype(np.float32) - z.astype(np.float32)[..., None]) * s.astype(np.float32)[..., None]
            assert torch.equal(torch.nan_to_num(got_x.cpu(), nan=7.0), torch.nan_to_num(torch.from_numpy(exact).to(out), nan=7.0))
            assert np.array_equal(np.isnan(got_x.float().cpu().numpy()), np.isnan(exact))


def test_slots_outside_the_cache_are_skipped_and_read_zero():
    from weight_only_int4_02_gb300 import w4a16
    cache = w4a16.kv4_cache(2, 2, 64, 16)
    k = torch.randn(4, 2, 64, device="cuda", dtype=torch.float16)
    slots = torch.tensor([-1, 5, 32, 1 << 40], device="cuda")
    w4a16.kv4_append(k, k, slots, cache, 16)
    other = w4a16.kv4_cache(2, 2, 64, 16)
    w4a16.kv4_append(k[1:2], k[1:2], slots[1:2], other, 16)
    assert torch.equal(cache, other)
    rk, rv = w4a16.kv4_read(cache, slots, 16)
    assert (rk[[0, 2, 3]] == 0).all() and (rv[[0, 2, 3]] == 0).all() and (rk[1] != 0).any()


def test_offsets_past_32_bits():
    from weight_only_int4_02_gb300 import w4a16
    page, D, heads = 256, 128, 2
    pages = (5 << 30) // w4a16.kv4_page_bytes(heads, D, page)
    cache = torch.empty((pages, heads, page // 16, 16 * (D + 6)), dtype=torch.uint8, device="cuda")
    k, v = (torch.randn(300, heads, D, device="cuda", dtype=torch.float16) for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    slots = torch.cat([torch.arange(256) + (pages - 1) * page, torch.arange(44) + (pages - 2) * page]).cuda()
    w4a16.kv4_append(k, v, slots, cache, page)
    small = w4a16.kv4_cache(2, heads, D, page)
    w4a16.kv4_append(k, v, torch.arange(300, device="cuda"), small, page)
    assert torch.equal(cache[pages - 1], small[0])
    q = torch.randn(1, 8, D, device="cuda", dtype=torch.float16)
    seq, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([300], [0, 1]))
    a = w4a16.kv4_attention(q, cache, table, seq, starts, page, 1)
    b = w4a16.kv4_attention(q, small, torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), seq, starts, page, 1)
    assert torch.equal(a, b)


# ---------------------------------------------------------------- attention
def batch_of(seq, nq, heads, group, D, page, dtype, seed, spread=0.3):
    """A cache filled through its definition, with NaN scales wherever no token is stored."""
    r = np.random.default_rng(seed)
    held = [-(-s // page) for s in seq]
    pages = sum(held) + 2
    ids = r.permutation(pages)
    cols = max(held + [1]) + 1
    table = np.full((len(seq), cols), -1, np.int32)
    cache = r.integers(0, 256, (pages, heads, page // 16, 16 * (D + 6)), dtype=np.uint8)
    cache[..., 16 * D:16 * D + 64] = np.array([0, 126], np.uint8).repeat(1).tolist() * 32   # binary16 NaN 0x7e00
    at = 0
    for b, s in enumerate(seq):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        for j in range(held[b]):
            live = min(page, s - j * page)
            blk = cache[table[b, j]]
            sc = np.exp(spread * r.standard_normal((heads, 2, page))) * 0.25
            sc[:, :, live:] = np.nan
            ze = r.integers(0, 16, (heads, 2, page)).astype(np.uint8)
            blk[:, :, 16 * D:16 * D + 32] = np.ascontiguousarray(sc[:, 0].reshape(heads, -1, 16).astype(np.float16)).view(np.uint8)
            blk[:, :, 16 * D + 32:16 * D + 64] = np.ascontiguousarray(sc[:, 1].reshape(heads, -1, 16).astype(np.float16)).view(np.uint8)
            blk[:, :, 16 * D + 64:16 * D + 80] = ze[:, 0].reshape(heads, -1, 16)
            blk[:, :, 16 * D + 80:] = ze[:, 1].reshape(heads, -1, 16)
    starts = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(starts[-1]), heads * group, D)) * 0.5).to(DT[dtype])
    return q, cache, table, np.array(seq, np.int32), starts


def check(q, cache, table, seq, starts, page, window, out, lse, scale=None):
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    o, l, smass, vmass = ref.attention(q.double().numpy(), cache, table, seq, starts, page, scale, window)
    # scores: FP32 sums of D products of q and bare codes, about one rounding of the running sum an MMA
    # (8 of 16 products), and the zero-point's share: 16 roundings of the mass at 2^-24 each
    es = 16 * 2.0 ** -24 * smass
    n = 2.0 ** -24 * (np.max(seq, initial=0) + 64)          # running sums over the keys
    # a probability's relative error: its score's twice over (its own and the maximum's) and the exponential's
    ep = (2 * es + 2.0 ** -21)[..., None] + n
    u = 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -8
    bound = u * np.abs(o) * 1.01 + vmass * ep * 2 + 2.0 ** -24
    got = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(o))
    err = np.where(np.isnan(o), 0.0, np.abs(got - o))
    assert (err <= np.where(np.isnan(o), 1.0, bound)).all(), "worst error over bound %.3f" % np.nanmax(err / bound)
    if lse is not None:
        g = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(g), np.isneginf(l)) and np.array_equal(np.isnan(g), np.isnan(l))
        f = np.isfinite(l)
        lim = (2 * es + 2.0 ** -21 + n + 2.0 ** -23 * np.abs(np.where(f, l, 0)))[f]
        assert (np.abs(g[f] - l[f]) <= lim).all()


def run(q, cache, table, seq, starts, page, window=0, **kw):
    from weight_only_int4_02_gb300 import w4a16
    max_q = int(np.max(np.diff(starts), initial=0))
    r = w4a16.kv4_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), page, max_q, window=window,
                            return_lse=True, **kw)
    assert w4a16.check_device_status() == w4a16.OK
    return r


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "float16"), (64, "bfloat16"), (128, "bfloat16")])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (2, 8), (1, 16), (1, 20)])
def test_decode_lengths(D, dtype, heads, group):
    seq = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 257, 700]
    nq = [1] * len(seq)
    for page, window in ((16, 0), (64, 0), (32, 40)):
        args = batch_of(seq, nq, heads, group, D, page, dtype, heads * 10 + group)
        check(*args, page, window, *run(*args, page, window))


@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
@pytest.mark.parametrize("heads,group,nq", [(2, 1, 5), (2, 4, 2), (1, 4, 4), (3, 2, 9), (1, 7, 33), (2, 1, 130), (1, 8, 70)])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_several_queries(D, dtype, heads, group, nq, window):
    seq = [nq, 0, 333, nq + 1, 200 + nq, 3]
    lens = [nq, 1, nq, max(1, nq - 3), 0, min(nq, 3)]
    args = batch_of(seq, lens, heads, group, D, 32, dtype, nq)
    check(*args, 32, window, *run(*args, 32, window))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("group,nq", [(4, 4), (3, 5), (8, 4), (4, 6)])
@pytest.mark.parametrize("window", [0, 50])
def test_batches_of_several_queries(D, dtype, group, nq, window):
    """Enough rows that segments of 16 are taken where they pay (12 to 16 and 32 rows a KV head, not 24)."""
    r = np.random.default_rng(group * nq)
    lens = r.integers(0, nq + 1, 96)
    lens[:3] = nq
    seq = lens + r.integers(0, 150, 96) * (r.random(96) < 0.9)
    seq[1], seq[2] = 777, max(0, nq - 2)
    args = batch_of([int(x) for x in seq], [int(x) for x in lens], 2, group, D, 16, dtype, nq)
    assert args[0].shape[0] * args[0].shape[1] > 1024
    out, lse = run(*args, 16, window)
    check(*args, 16, window, out, lse)
    # a poisoned token shows in the row that sees it alone, a missing page hides its tokens
    q, cache, table, seq, starts = args
    t = int(seq[1]) - 1
    cache[table[1, t // 16], 1, 0, 16 * D + 32 + 2 * (t % 16):][:2] = [0, 126]
    table[0, 0] = -1
    out, _ = run(*args, 16, window)
    check(*args, 16, window, out, None)
    bad = torch.isnan(out).any(-1)
    assert bad[2 * nq - 1, group:].all() and int(bad.sum()) == group


@pytest.mark.parametrize("D", [64, 128])
def test_more_queries_than_tokens_leave_rows_empty(D):
    args = batch_of([3, 40], [9, 3], 2, 2, D, 16, "float16", 5)
    out, lse = run(*args, 16)
    check(*args, 16, 0, out, lse)
    assert (out[:6] == 0).all() and torch.isneginf(lse[:6]).all()


def test_one_long_request_is_split_over_the_gpu():
    args = batch_of([20011], [1], 2, 4, 128, 64, "float16", 3)
    out, lse = run(*args, 64)
    check(*args, 64, 0, out, lse)
    again, _ = run(*args, 64)
    assert torch.equal(out, again)


@pytest.mark.parametrize("spread", [3.0])
def test_scales_of_many_sizes(spread):
    args = batch_of([900, 31], [1, 1], 2, 4, 128, 16, "float16", 9, spread=spread)
    check(*args, 16, 0, *run(*args, 16))


def test_missing_pages_hide_their_tokens():
    q, cache, table, seq, starts = batch_of([200, 100], [1, 2], 2, 2, 64, 16, "float16", 4)
    table[0, 3], table[0, 7], table[1, 0] = -1, cache.shape[0] + 5, -7
    check(q, cache, table, seq, starts, 16, 0, *run(q, cache, table, seq, starts, 16))
    table[:] = -1      # every row of every request empty
    out, lse = run(q, cache, table, seq, starts, 16)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("nq", [2, 20])
def test_a_poisoned_token_shows_where_it_is_seen_and_nowhere_else(nq):
    for which in (0, 1):       # K's scale, V's scale
        q, cache, table, seq, starts = batch_of([60, 50], [nq, 1], 1, 4, 128, 16, "bfloat16", 4)
        t = 59                 # the last token of request 0: its last query alone sees it
        cache[table[0, t // 16], 0, 0, 16 * 128 + 32 * which + 2 * (t % 16):][:2] = [0, 126]
        out, lse = run(q, cache, table, seq, starts, 16)
        check(q, cache, table, seq, starts, 16, 0, out, lse if which == 0 else None)
        assert torch.isnan(out[nq - 1]).all() and not torch.isnan(out[:nq - 1]).any() and not torch.isnan(out[nq:]).any()


def test_large_and_small_queries():
    q, cache, table, seq, starts = batch_of([100, 77, 30], [1, 1, 1], 1, 8, 128, 16, "bfloat16", 6)
    q[0] *= 60.0
    q[1] *= 1e-20
    q[2] = 0
    check(q, cache, table, seq, starts, 16, 0, *run(q, cache, table, seq, starts, 16))


def test_strided_views_streams_and_workspaces():
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([90, 700, 3], [2, 2, 1], 2, 4, 128, 32, "float16", 8)
    want, want_lse = run(q, cache, table, seq, starts, 32)
    T, H, D = q.shape
    wide = torch.zeros((T, H + 4, D + 8), dtype=q.dtype)
    wide[:, 2:2 + H, :D] = q
    view = wide.cuda()[:, 2:2 + H, :D]
    out = torch.full((T, H + 1, D + 16), 9.0, dtype=q.dtype, device="cuda")
    wide_table = cuda(np.concatenate([table, np.full_like(table, 1 << 30)], 1))[:, :table.shape[1]]
    ws = torch.zeros(w4a16.kv4_workspace_bytes(), dtype=torch.uint8, device="cuda")
    c, sl, st = cuda(cache), cuda(seq), cuda(starts)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got, lse = w4a16.kv4_attention(view, c, wide_table, sl, st, 32, 2, out=out[:, 1:, :D], return_lse=True, workspace=ws,
                                   stream=stream)
    stream.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    assert (out[:, 0] == 9.0).all() and (out[:, :, D:] == 9.0).all()
    # another scale
    got, lse = w4a16.kv4_attention(view, c, wide_table, sl, st, 32, 2, scale=0.25, return_lse=True)
    check(q, cache, table, seq, starts, 32, 0, got, lse, scale=0.25)
    # captured into a graph, replayed on new lengths
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4a16.kv4_attention(view, c, wide_table, sl, st, 32, 2, out=out[:, 1:, :D], workspace=ws)
    sl.copy_(cuda(np.array([40, 500, 2], np.int32)))
    g.replay()
    torch.cuda.synchronize()
    check(q, cache, table, np.array([40, 500, 2], np.int32), starts, 32, 0, out[:, 1:, :D], None)


def test_max_q_only_chooses_the_kernel():
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([90, 200], [3, 40], 1, 4, 64, 16, "bfloat16", 8)
    for max_q in (0, 1, 4, 1000):
        out = w4a16.kv4_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), 16, max_q)
        check(q, cache, table, seq, starts, 16, 0, out, None)


def test_a_step_from_lengths_to_output():
    """Tables, append and attention chained, two steps, against attention over the quantised rows."""
    from weight_only_int4_02_gb300 import w4a16
    heads, group, D, page = 2, 4, 128, 16
    cache = w4a16.kv4_cache(40, heads, D, page)
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(40, device="cuda").to(torch.int32)
    taken, seq = None, np.zeros(3, np.int32)
    for new in ([20, 1, 33], [1, 1, 1]):
        seq = seq + np.array(new, np.int32)
        T = sum(new)
        q = torch.randn(T, heads * group, D, device="cuda", dtype=torch.float16)
        k, v = (torch.randn(T, heads, D, device="cuda", dtype=torch.float16) for _ in range(2))
        sl = cuda(seq)
        slots, _, starts, taken = w4a16.kv4_tables(sl, cuda(np.array(new, np.int32)), free, table, page, T, taken=taken)
        w4a16.kv4_append(k, v, slots, cache, page)
        out, lse = w4a16.kv4_attention(q, cache, table, sl, starts, page, max(new), return_lse=True)
        check(q.cpu(), cache.cpu().numpy(), table.cpu().numpy(), seq, starts.cpu().numpy(), page, 0, out, lse)
