"""The 4-bit key-value cache's calls at the ends of their arguments' ranges, against their definitions.

Both attention kernels are forced in turn. The stream-K kernel is held to the tolerance derived in test_kv4_gpu.py; the
tcgen05 kernel, as in test_kv4_prompt_gpu.py, to that and its rounding of probabilities times V's scale to binary16 for
bfloat16 outputs: a relative 2^-11 of sum p |v|, here bounded by sum p s (c + z)."""
import numpy as np
import pytest

from tests import serving_reference as ref
from tests.test_kv4_gpu import batch_of, check, cuda, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("D", [64, 128])
def test_bfloat16_rows_past_the_largest_scale(D):
    """Rows of magnitudes 2^15 to 2^126, where the scale stays at 65504: every code is the formula's, exactly."""
    from weight_only_int4_02_gb300 import w4a16
    r = np.random.default_rng(D)
    exps = np.arange(15.0, 126.0, 0.25)
    x = r.standard_normal((len(exps), 2, D)) * np.exp2(exps)[:, None, None]
    x[:, 1] = -np.abs(x[:, 1])                       # one sign only: zero-point 15
    x[:, 0, ::3] = r.standard_normal((len(exps), len(range(0, D, 3)))) * 1e5   # beside values that the scale holds
    x[:, 0, 0] = -np.exp2(exps)                      # below zero under a zero-point of its own
    k = torch.from_numpy(x).to(torch.bfloat16)
    v = -k
    pages = -(-len(exps) // 16)
    cache = w4a16.kv4_cache(pages, 2, D, 16)
    slots = torch.arange(len(exps), device="cuda")
    w4a16.kv4_append(k.cuda(), v.cuda(), slots, cache, 16)
    with np.errstate(over="ignore"):
        for got, y in zip(w4a16.kv4_read(cache, slots, 16, dtype=torch.float32), (k, v)):
            code, scale, zero = ref.quantise(y.float().numpy())
            want = (code.astype(np.float32) - zero[..., None]) * scale.astype(np.float32)[..., None]
            assert np.array_equal(got.cpu().numpy(), want)


def on_path(path, args, page, window, oracle_table=None):
    """One call on the forced kernel, checked; oracle_table: what the oracle reads instead of the table given."""
    from weight_only_int4_02_gb300 import w4a16
    before = w4a16.kv4_force_path(path)
    try:
        out, lse = run(*args, page, window)
    finally:
        w4a16.kv4_force_path(before)
    q, cache, table, seq, starts = args
    table = table if oracle_table is None else oracle_table
    if path == 1 or q.dtype == torch.float16:        # two binary16 parts, 2^-21: within the tolerance's own terms
        check(q, cache, table, seq, starts, page, window, out, lse)
    else:
        o, l, smass, vmass = ref.attention(q.double().numpy(), cache, table, seq, starts, page, q.shape[-1] ** -0.5, window)
        es, n = 16 * 2.0 ** -24 * smass, 2.0 ** -24 * (np.max(seq, initial=0) + 64)
        ep = (2 * es + 2.0 ** -21)[..., None] + n
        err = np.abs(out.double().cpu().numpy() - o)
        assert (err <= 2.0 ** -8 * 1.01 * np.abs(o) + vmass * (2 * ep + 2.0 ** -11) + 2.0 ** -24).all()
        g, f = lse.double().cpu().numpy(), np.isfinite(l)
        assert np.array_equal(np.isfinite(g), f)
        assert (np.abs(g[f] - l[f]) <= (2 * es + 2.0 ** -21 + n + 2.0 ** -23 * np.abs(np.where(f, l, 0)))[f]).all()
    return out, lse


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
def test_the_largest_window_hides_nothing(path, D, dtype):
    """A window of 2^31 - 1 is no window, also where a request has more queries than cached tokens."""
    args = batch_of([3, 40, 130, 0, 700], [9, 60, 1, 3, 50], 2, 4, D, 16, dtype, 5)
    out, lse = on_path(path, args, 16, 2 ** 31 - 1)
    want, want_lse = on_path(path, args, 16, 0)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("window", [0, 20, 300])
def test_requests_longer_than_their_table(path, D, dtype, window):
    """Tokens past the table's columns are hidden; the queries' positions still count them."""
    q, cache, table, seq, starts = batch_of([480, 512, 100, 400], [70, 1, 40, 33], 2, 4, D, 16, dtype, 7)
    seq = seq + np.array([60, 20, 0, 900], np.int32)   # the last request's window, where it has one, lies past its table
    cols = 30                                          # 480 tokens
    wide = np.full((4, 90), -1, np.int32)
    wide[:, :cols] = table[:, :cols]
    out, lse = on_path(path, (q, cache, wide[:, :cols], seq, starts), 16, window, oracle_table=wide)
    assert window == 0 or (out[starts[3]:] == 0).all()


@pytest.mark.parametrize("new", [[8191], [1, 3000, 0, 777, 129, 128]])
def test_tables_of_long_chunks(new):
    from weight_only_int4_02_gb300 import w4a16
    r = np.random.default_rng(len(new))
    page = 32
    new = np.array(new, np.int32)
    seq = new + r.integers(0, 5000, len(new)).astype(np.int32)
    cols = int(-(-seq.max() // page)) - 3            # the longest request ends past its row
    free = r.permutation(4000).astype(np.int32)
    held = r.integers(0, 4000, (len(new), cols)).astype(np.int32)
    want = ref.tables(seq, new, free, held, page, 0)
    table = cuda(held)
    slots, positions, starts, taken = w4a16.kv4_tables(cuda(seq), cuda(new), cuda(free), table, page, int(new.sum()))
    assert np.array_equal(table.cpu().numpy(), want[0]) and slots.tolist() == want[1] and positions.tolist() == want[2]
    assert starts.tolist() == want[3] and taken.item() == want[4]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_a_request_of_a_hundred_thousand_tokens(dtype):
    args = batch_of([100003], [2], 1, 4, 128, 256, dtype, 11)
    check(*args, 256, 0, *run(*args, 256))


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("group,nq", [(4, 1), (8, 1), (8, 2)])
def test_long_sums_have_no_bias(D, dtype, group, nq):
    """512 requests over one row of 16384 tokens, so that each warp sums about a hundred units of 32 tokens or more.
    An MMA rounds towards zero. If a unit's two tiles, each with a high and a low part, add its share of sum p s c to sums
    of either sign, and then sum p s z is taken off, the roundings lose less than 2^-23 of half and of all of that share,
    twice, 2^-24 on average: 3 * 2^-24 of the whole mass. Outputs are rounded to nearest, which has no bias: five
    deviations of their mean."""
    from weight_only_int4_02_gb300 import w4a16
    n, seq, page = 512, 16384, 256
    _, cache, table, _, _ = batch_of([seq], [1], 1, group, D, page, dtype, D + group)
    g = torch.Generator(device="cuda").manual_seed(group)
    q = torch.randn(n * nq, group, D, generator=g, device="cuda").to(getattr(torch, dtype))
    rows = cuda(table).expand(n, -1)
    lens = torch.full((n,), seq, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, n * nq + 1, nq, dtype=torch.int32, device="cuda")
    before = w4a16.kv4_force_path(1)
    try:
        out = w4a16.kv4_attention(q, cuda(cache), rows, lens, starts, page, nq).double()
    finally:
        w4a16.kv4_force_path(before)
    kc, ks, kz, vc, vs, vz = [torch.from_numpy(x[:seq].astype(np.float64)).cuda()
                              for x in ref.decode(cache[table[0, :seq // page], 0].reshape(-1, 16 * (D + 6)), D)]
    x = q.double().view(n, nq, group, D) @ ((kc - kz[:, None]) * ks[:, None]).T * D ** -0.5
    pos = torch.arange(seq - nq, seq, device="cuda")[None, :, None, None]
    p = torch.softmax(x.masked_fill(torch.arange(seq, device="cuda") > pos, -np.inf), -1).view(-1, seq)
    o = (p @ ((vc - vz[:, None]) * vs[:, None])).view(out.shape)
    mass = float((p @ (vs * vc.amax(-1))).mean())    # sum p s c, with the largest code of each token
    u = 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
    noise = 5 * u * float(o.square().mean().sqrt()) / 3 ** 0.5 / out.numel() ** 0.5
    bias = float((out - o).mean())
    assert abs(bias) <= 3 * 2.0 ** -24 * mass + noise, (bias, mass, noise)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("batch,nq", [(1000, 2), (70, 40)])
def test_batches_of_many_requests(path, batch, nq):
    """More requests than a CTA has threads, and than a warp looks at together; lengths and queries of every size, none too."""
    r = np.random.default_rng(batch)
    lens = r.integers(0, nq + 1, batch)
    seq = (lens + r.integers(0, 60, batch)) * (r.random(batch) < 0.9)
    args = batch_of([int(x) for x in seq], [int(x) for x in lens], 1, 4, 64, 16, "float16", batch)
    on_path(path, args, 16, 0)
