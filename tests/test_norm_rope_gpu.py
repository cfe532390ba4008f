"""Norms of queries and keys and their rotation on the GPU against the definition in 64 bits.

Tolerance: the output's rounding, half a step of its size; in FP32 the sum of squares of D = 64 or 128 values (a chain of 8
multiply-adds and at most 4 sums: 12 roundings of 2^-24, halved by the root), the root's reciprocal (two units of 2^-23), two products,
and the rotation's two products and a sum, of |a cos| + |b sin|: below 2^-20 of that mass altogether. Binary16 outputs below 2^-14 are
rounded to multiples of 2^-24."""
import numpy as np
import pytest

from tests import kv8_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def expected(x, w, eps, positions, table, interleaved):
    """(y, mass) float64 of x [tokens][heads][D], w [D] or None, table or None."""
    x = x.double().cpu().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.double().cpu().numpy()
    if table is None:
        return x, np.abs(x)
    cos, sin = np.abs(table[:, :table.shape[1] // 2]), np.abs(table[:, table.shape[1] // 2:])
    plus = np.concatenate([cos, -sin], 1)       # |a| cos + |b| sin by the rotation with -sin, |b| cos + |a| sin with +sin
    a, b = (ref.rotate(np.abs(x), positions, t, interleaved) for t in (plus, np.concatenate([cos, sin], 1)))
    return ref.rotate(x, positions, table, interleaved), np.maximum(np.abs(a), np.abs(b))


def close(got, want, mass, dtype):
    got = got.double().cpu().numpy()
    u, least = (2.0 ** -11, 2.0 ** -25) if dtype == torch.float16 else (2.0 ** -8, 2.0 ** -134)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    err = np.abs(got - want) - (u * np.abs(want) + 2.0 ** -20 * mass * (1 + u) + least)
    assert np.nanmax(err, initial=-1) <= 0


def inputs(tokens, heads, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, D, generator=g) * torch.exp(torch.randn(tokens, heads, 1, generator=g))
    x[0] = 0.0
    x[-1] *= 2.0 ** -12
    return x.to(dtype)


@pytest.mark.parametrize("D,dtype", [(64, "float16"), (64, "bfloat16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("tokens,q_heads,kv_heads", [(1, 1, 1), (3, 7, 1), (17, 8, 8), (130, 28, 4), (5, 64, 8), (2, 33, 0), (9, 0, 3)])
@pytest.mark.parametrize("rot,interleaved,norm", [(None, False, True), ("all", False, True), ("all", True, False), (16, False, False),
                                                  (24, True, True), (40, False, True)])
def test_norms_and_rotation(D, dtype, tokens, q_heads, kv_heads, rot, interleaved, norm):
    from weight_only_int4_02_gb300 import w4a16
    dt = DT[dtype]
    r = np.random.default_rng(tokens)
    rot = D if rot == "all" else rot
    table = None if rot is None else ref.rope_table(5000, rot)
    pos = None if rot is None else r.integers(0, 5000, tokens).astype(np.int32)
    q = inputs(tokens, q_heads, D, dt, 1) if q_heads else None
    k = inputs(tokens, kv_heads, D, dt, 2) if kv_heads else None
    wq, wk = ((1 + 0.3 * torch.randn(D)).to(dt) if norm and x is not None else None for x in (q, k))
    up = lambda t: None if t is None else t.cuda() if torch.is_tensor(t) else torch.from_numpy(t).cuda()
    out = w4a16.qk_norm_rope(up(q), up(k), up(pos), up(table), q_weight=up(wq), k_weight=up(wk), eps=1e-5, interleaved=interleaved)
    for got, x, w in zip(out, (q, k), (wq, wk)):
        if x is None:
            assert got is None
            continue
        assert got.shape == x.shape and got.dtype == dt and got.is_contiguous()
        close(got, *expected(x, w, 1e-5, pos, table, interleaved), dt)


def test_one_weight_alone_and_an_eps_that_counts():
    from weight_only_int4_02_gb300 import w4a16
    q, k = inputs(6, 4, 128, torch.bfloat16, 1), inputs(6, 2, 128, torch.bfloat16, 2)
    w = torch.ones(128, dtype=torch.bfloat16)
    a, b = w4a16.qk_norm_rope(q.cuda(), k.cuda(), q_weight=w.cuda(), eps=0.5)
    close(a, *expected(q, w, 0.5, None, None, False), q.dtype)
    assert torch.equal(b.cpu(), k)
    a, b = w4a16.qk_norm_rope(q.cuda(), k.cuda(), k_weight=w.cuda(), eps=0.5)
    assert torch.equal(a.cpu(), q)
    close(b, *expected(k, w, 0.5, None, None, False), q.dtype)


def test_padding_stays_and_positions_past_the_table_show():
    from weight_only_int4_02_gb300 import w4a16
    table = torch.from_numpy(ref.rope_table(50, 64)).cuda()
    q, k = inputs(6, 4, 64, torch.float16, 1).cuda(), inputs(6, 2, 64, torch.float16, 2).cuda()
    pos = torch.tensor([3, -1, 49, 50, 1 << 30, -(1 << 31)], dtype=torch.int32, device="cuda")
    mark = [torch.full_like(x, 9.0) for x in (q, k)]
    out = w4a16.qk_norm_rope(q, k, pos, table, q_out=mark[0], k_out=mark[1])
    fine = w4a16.qk_norm_rope(q, k, pos.clamp(0, 49), table)
    for a, m, f in zip(out, mark, fine):
        assert a.data_ptr() == m.data_ptr()
        assert torch.equal(a[[0, 2]], f[[0, 2]]) and (a[[1, 5]] == 9.0).all() and torch.isnan(a[[3, 4]]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 24])
def test_slices_in_place_on_a_stream_and_captured(rot, interleaved):
    from weight_only_int4_02_gb300 import w4a16
    T, H, KV, D = 37, 12, 4, 64
    x = inputs(T, H + 2 * KV + 1, D, torch.bfloat16, 3).cuda()
    table = w4a16.rope_table(300, rot)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7
    w = (1 + 0.1 * torch.randn(2, D, device="cuda")).to(torch.bfloat16)
    args = dict(positions=pos, rope=table, q_weight=w[0].clone(), k_weight=w[1].clone(), interleaved=interleaved)
    split = lambda y: (y[:, 1:H + 1], y[:, H + 1:H + 1 + KV])
    want = w4a16.qk_norm_rope(*split(x), **args)
    y, z = x.clone(), x.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = w4a16.qk_norm_rope(*split(y), q_out=split(y)[0], k_out=split(y)[1], stream=s, **args)
    fresh = w4a16.qk_norm_rope(*split(z), stream=s, **args)
    s.synchronize()
    for a, b, c in zip(got, want, fresh):
        assert torch.equal(a, b) and torch.equal(c, b)
    assert torch.equal(y[:, 0], x[:, 0]) and torch.equal(y[:, H + 1 + KV:], x[:, H + 1 + KV:]) and torch.equal(z, x)
    g = torch.cuda.CUDAGraph()
    out = [torch.zeros_like(t) for t in want]
    with torch.cuda.graph(g):
        w4a16.qk_norm_rope(*split(z), q_out=out[0], k_out=out[1], **args)
    pos.add_(3)
    g.replay()
    for a, b in zip(out, w4a16.qk_norm_rope(*split(z), **args)):
        assert torch.equal(a, b) and not torch.equal(a, want[0][:, :0])


def test_infinities_and_nans_stay_in_their_rows():
    from weight_only_int4_02_gb300 import w4a16
    q = inputs(4, 8, 128, torch.float16, 1)
    q[1, 2, 5], q[3, 7, 100] = np.inf, np.nan
    w = torch.ones(128, dtype=torch.float16).cuda()
    got, _ = w4a16.qk_norm_rope(q.cuda(), None, torch.arange(4, dtype=torch.int32).cuda(), w4a16.rope_table(4, 128), q_weight=w)
    bad = torch.isnan(got).any(-1).cpu()
    assert bad[1, 2] and bad[3, 7] and int(bad.sum()) == 2


def test_many_tokens_and_heads():
    """Every row is written once: 70000 tokens, and 1000 heads."""
    from weight_only_int4_02_gb300 import w4a16
    for T, H, KV, D in ((70001, 3, 1, 64), (3, 1000, 17, 128)):
        q, k = (torch.randn(T, n, D, device="cuda").to(torch.float16) for n in (H, KV))
        table = w4a16.rope_table(16, D)
        pos = (torch.arange(T, device="cuda") % 16).to(torch.int32)
        for x, y in zip((q, k), w4a16.qk_norm_rope(q, k, pos, table)):
            at = table[pos.long()].double()[:, None]
            a, b = x.double().chunk(2, -1)
            cos, sin = at.chunk(2, -1)
            want = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            assert ((y.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -20 * 8 + 2.0 ** -25).all()


@pytest.mark.parametrize("rows,rot,base", [(1, 8, 10000.0), (3000, 24, 500000.0), (70000, 128, 10000.0)])
def test_the_table_is_rounded_once(rows, rot, base):
    """Angles in 64 bits: at position 70000 an angle is 2^-36 off at most, far below half a step of its cosine."""
    from weight_only_int4_02_gb300 import w4a16
    got = w4a16.rope_table(rows, rot, base).double().cpu().numpy()
    angle = np.arange(rows)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    want = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -34).all()


def test_no_tokens():
    from weight_only_int4_02_gb300 import w4a16
    z = torch.zeros(0, 4, 64, dtype=torch.float16, device="cuda")
    a, b = w4a16.qk_norm_rope(z, z[:, :2], torch.zeros(0, dtype=torch.int32, device="cuda"), w4a16.rope_table(4, 64))
    assert a.shape == z.shape and b.shape == (0, 2, 64)


def test_refusals():
    from weight_only_int4_02_gb300 import w4a16
    from tests.test_binding_refusals_gpu import every_other, refused
    q, k = (torch.randn(5, n, 64, device="cuda").to(torch.float16) for n in (4, 2))
    pos, table = torch.arange(5, dtype=torch.int32, device="cuda"), w4a16.rope_table(9, 64)
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    odd = torch.zeros(5, 4, 68, dtype=torch.float16, device="cuda")
    wide = torch.zeros(5, 4, 72, dtype=torch.float16, device="cuda")
    refused(w4a16.qk_norm_rope, dict(q=q, k=k, positions=pos, rope=table, q_weight=w, k_weight=w, q_out=q.clone(), k_out=k.clone()), [
        ("q", q.float()), ("q", q.bfloat16()), ("q", q[:4]), ("q", q[0]), ("q", q[..., :32]), ("q", every_other(q)), ("q", odd[..., :64]),
        ("q", wide[..., 1:65]), ("q", q[:1].expand(5, -1, -1)), ("q", q.cpu()), ("q", None), ("k", k.bfloat16()), ("k", k[:3]),
        ("k", k.cpu()), ("k", every_other(k)), ("k", None), ("positions", None), ("positions", pos.long()), ("positions", pos[:4]),
        ("positions", every_other(pos)), ("positions", pos.cpu()), ("rope", None), ("rope", table.double()), ("rope", table[0]),
        ("rope", table[:, :20].contiguous()), ("rope", table.t().contiguous().t()), ("rope", w4a16.rope_table(9, 72)), ("rope", table[:0]),
        ("rope", table.cpu()), ("q_weight", w.float()), ("q_weight", w[:32]), ("q_weight", every_other(w)), ("k_weight", w[None]),
        ("k_weight", w.cpu()), ("q_out", k.clone()), ("q_out", q.float()), ("q_out", every_other(q)), ("q_out", odd[..., :64]),
        ("k_out", q.clone()), ("k_out", k.cpu()), ("eps", -1.0), ("eps", float("nan")), ("eps", "x")])
    with pytest.raises(w4a16.W4A16Error):
        w4a16.qk_norm_rope(None, None, pos, table)
    with pytest.raises(w4a16.W4A16Error):
        w4a16.qk_norm_rope(q, None, pos, table, k_weight=w)
    with pytest.raises(w4a16.W4A16Error):
        w4a16.rope_table(4, 12)
