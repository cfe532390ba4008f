"""Attention of prompt chunks over the 4-bit cache by the tcgen05 kernel (forced where the
dispatcher would leave so few rows to the stream-K kernel) against its definition in 64 bits, over
several row tiles and blocks of cached tokens.

Tolerance, beside what test_kv4_gpu.py derives for scores and sums: probabilities times V's scale are
rounded to binary16 once (2^-12 each side of a half step: a relative 2^-11 of sum p |v| bounds it) when
outputs are bfloat16; outputs in binary16 get a second, low part, which leaves 2^-21."""
import numpy as np
import pytest

from tests import serving_reference as ref
from tests.test_kv4_gpu import DT, batch_of, cuda

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from weight_only_int4_02_gb300 import w4a16
    before = w4a16.kv4_force_path(2)
    yield
    w4a16.kv4_force_path(before)


def value_mass(q, cache, table, seq, starts, page, scale, window):
    """sum p |v| / sum p, per output value."""
    T, H, D = q.shape
    kv = cache.shape[1]
    g = H // kv
    out = np.zeros((T, H, D))
    for b in range(len(seq)):
        n, a, e = int(seq[b]), int(starts[b]), int(starts[b + 1])
        ids = table[b, :-(-n // page)]
        for h in range(kv):
            if n == 0:
                continue
            kc, ks, kz, vc, vs, vz = [x[:n].astype(np.float64) for x in ref.decode(cache[ids, h].reshape(-1, 16 * (D + 6)), D)]
            key, val = (kc - kz[:, None]) * ks[:, None], np.abs((vc - vz[:, None]) * vs[:, None])
            pos, col = np.arange(n - (e - a), n)[:, None], np.arange(n)[None]
            see = (col <= pos) & ((col > pos - window) if window > 0 else True)
            for j in range(h * g, (h + 1) * g):
                x = np.where(see, q[a:e, j] @ key.T * scale, -np.inf)
                m = x.max(-1, keepdims=True)
                p = np.exp(x - np.where(np.isneginf(m), 0, m))
                l = p.sum(-1, keepdims=True)
                out[a:e, j] = p @ val / np.where(l == 0, 1, l)
    return out


def run_and_check(args, page, window=0, scale=None, **kw):
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = args
    D = q.shape[-1]
    sc = D ** -0.5 if scale is None else scale
    max_q = int(np.diff(starts).max())
    out, lse = w4a16.kv4_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), page, max_q, window=window,
                                   scale=scale, return_lse=True, **kw)
    assert w4a16.check_device_status() == w4a16.OK
    q64 = q.double().numpy()
    o, l, smass, vmass = ref.attention(q64, cache, table, seq, starts, page, sc, window)
    fed = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -21
    es = 16 * 2.0 ** -24 * np.abs(smass)
    n = 2.0 ** -24 * (np.max(seq) + 64)
    u = 2.0 ** -11 if q.dtype == torch.float16 else 2.0 ** -8
    bound = (u * 1.01 * np.abs(o) + vmass * 2 * ((2 * es + 2.0 ** -21)[..., None] + n) +
             fed * value_mass(q64, cache, table, seq, starts, page, sc, window) + 2.0 ** -24)
    err = np.abs(out.double().cpu().numpy() - o)
    assert (err <= bound).all(), "worst error over bound %.3f" % np.nanmax(err / bound)
    g, f = lse.double().cpu().numpy(), np.isfinite(l)
    assert np.array_equal(np.isneginf(g), ~f)
    assert (np.abs(g - l)[f] <= (2 * es + 2.0 ** -21 + n + 2.0 ** -23 * np.abs(np.where(f, l, 0)))[f]).all()
    return out, lse


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (64, "bfloat16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("heads,group,lens,seq", [
    (1, 4, [150, 33], [700, 33]),          # three row tiles with a ragged one, blocks behind cached context
    (2, 1, [300, 1, 40], [300, 900, 1000]),   # one head a group; a decode row in the same batch
    (1, 8, [64], [128]), (1, 8, [65], [129]), (1, 3, [100], [383])])
@pytest.mark.parametrize("window", [0, 129])
def test_prompt_chunks(D, dtype, heads, group, lens, seq, window):
    run_and_check(batch_of(seq, lens, heads, group, D, 32, dtype, sum(lens) + D), 32, window)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_page_sizes_and_a_small_window(page):
    args = batch_of([600, 90], [200, 90], 1, 2, 128, page, "bfloat16", page)
    run_and_check(args, page, window=7)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_scales_that_grow_along_the_tokens(dtype):
    """V's scales and the scores rise block after block: outputs and sums are rescaled on the way."""
    args = batch_of([900], [60], 1, 2, 128, 16, dtype, 5, spread=0.0)
    q, cache, table, seq, starts = args
    D = 128
    for t in range(900):
        at = cache[table[0, t // 16], 0, 0]
        for off, rise in ((16 * D, 1 / 150), (16 * D + 32, 1 / 60)):
            v = np.float16(0.02 * 2.0 ** (t * rise))
            at[off + 2 * (t % 16):off + 2 * (t % 16) + 2] = np.frombuffer(v.tobytes(), np.uint8)
    run_and_check(args, 16)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_other_softmax_scales(scale):
    run_and_check(batch_of([300], [80], 1, 2, 64, 16, "float16", 9), 16, scale=scale)
    run_and_check(batch_of([300], [2], 1, 2, 64, 16, "float16", 9), 16, scale=scale)


def test_missing_pages_and_poisoned_tokens():
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([400], [100], 1, 4, 128, 16, "bfloat16", 4)
    D = 128
    table[0, 3], table[0, 9] = -1, cache.shape[0] + 3
    call = lambda: w4a16.kv4_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), 16, 100, return_lse=True)
    out, lse = call()
    o, l, _, vmass = ref.attention(q.double().numpy(), cache, table, seq, starts, 16, D ** -0.5, 0)
    assert (np.abs(out.double().cpu().numpy() - o) <= 2.0 ** -8 * 1.01 * np.abs(o) + 2.0 ** -10 * vmass).all()
    for which in (0, 1):       # K's scale, then V's: seen by the last 30 queries alone
        bad = cache.copy()
        t = 370
        bad[table[0, t // 16], 0, 0, 16 * D + 32 * which + 2 * (t % 16):][:2] = [0, 126]
        good, cache = cache, bad
        got, got_lse = call()
        cache = good
        assert torch.isnan(got[70:]).all() and torch.equal(got[:70], out[:70])
        assert torch.isnan(got_lse[70:]).all() if which == 0 else torch.equal(got_lse, lse)


@pytest.mark.parametrize("path", [0, 1, 2])
def test_every_path_serves_a_batch_of_prompts_and_decodes(path):
    from weight_only_int4_02_gb300 import w4a16
    w4a16.kv4_force_path(path)
    # 7500 rows over eight query heads: the dispatcher's own choice is the tcgen05 kernel with the stream-K one
    run_and_check(batch_of([940, 300, 65, 0], [900, 1, 38, 1], 2, 4, 128, 64, "bfloat16", 3), 64)


def test_repeats_are_the_same_and_strided_views_too():
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([500, 77], [120, 77], 2, 4, 128, 32, "float16", 8)
    a = [cuda(x) for x in (cache, table, seq, starts)]
    T, H, D = q.shape
    wide = torch.zeros((T, H + 3, D + 8), dtype=q.dtype)
    wide[:, 1:1 + H, :D] = q
    out = torch.full((T, H + 1, D), 7.0, dtype=q.dtype, device="cuda")
    first = w4a16.kv4_attention(q.cuda(), *a, 32, 120)
    w4a16.kv4_attention(wide.cuda()[:, 1:1 + H, :D], *a, 32, 120, out=out[:, 1:])
    assert torch.equal(out[:, 1:], first) and (out[:, 0] == 7.0).all()


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (64, "bfloat16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("heads,group,lens,seq", [(2, 4, [40], [3000]), (1, 3, [150, 30], [2500, 1150]), (1, 8, [64], [1024])])
@pytest.mark.parametrize("window", [0, 1300])
def test_cached_tokens_are_split_over_several_ctas(D, dtype, heads, group, lens, seq, window):
    """Few row tiles over many tokens: the parts of a tile are joined, rows that see nothing in a part among them."""
    args = batch_of(seq, lens, heads, group, D, 64, dtype, sum(seq) + D)
    out, lse = run_and_check(args, 64, window)
    again, lse_again = run_and_check(args, 64, window)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


def test_a_poisoned_token_of_one_part_shows_in_the_rows_that_see_it():
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([2000], [100], 1, 4, 128, 16, "bfloat16", 4)
    D, t = 128, 700
    cache[table[0, t // 16], 0, 0, 16 * D + 32 + 2 * (t % 16):][:2] = [0, 126]
    table[0, 100] = -1     # a missing page hides what it holds
    for window, rows in ((0, 100), (1250, 50)):     # the first 50 queries see position 700: 1900 + i - 1250 < 700
        out = w4a16.kv4_attention(q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), 16, 100, window=window)
        assert torch.isnan(out[:rows]).all() and not torch.isnan(out[rows:]).any()
