"""Sampling on the GPU against its definition in 64 bits, and exactly where the weights are known."""
import numpy as np
import pytest

from tests import serving_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
F = np.float32


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def sample(x, u, temperature, top_k, top_p, min_p, strided=0):
    from weight_only_int4_02_gb300 import w4a16
    if strided:
        wide = torch.full((x.shape[0], x.shape[1] + strided), 99.0, dtype=x.dtype)
        wide[:, 1:1 + x.shape[1]] = x
        x = wide.cuda()[:, 1:1 + x.shape[1]]
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a).astype(d)).cuda()
    token, prob = w4a16.sample(x.cuda(), t(u, F), t(temperature, F), t(top_k, np.int32), t(top_p, F), t(min_p, F))
    return token.cpu().numpy(), prob.cpu().numpy()


def check(x, u, temperature, top_k, top_p, min_p, token, prob):
    """The drawn token against the row's draw in float64. A weight is off by at most 2^-32 (its rounding) and,
    relatively, by |y| 2^-23 for the exponent's roundings (|y| < 23) and 2^-22 for the exponential: below 4e-6.
    A token may be kept or not where the limit is that near; the drawn place moves by no more than the weights."""
    for b in range(x.shape[0]):
        row = x[b].double().numpy()
        n = len(row)
        if not (np.nan_to_num(row, nan=-np.inf) > -np.inf).any():
            assert token[b] == -1 and prob[b] == 0
            continue
        rank, e, keep, before = ref.sample_row(row, u[b], F(temperature[b]), top_k[b], F(top_p[b]), F(min_p[b]))
        tol = 4e-6 + n * 2.0 ** -32 / e[keep].sum()
        i = token[b]
        assert 0 <= i < n and keep[i], (b, i)
        sure = keep & (before < F(top_p[b]) - tol) & (e >= F(min_p[b]) * (1 + tol))
        maybe = keep & (before < F(top_p[b]) + tol) & (e >= F(min_p[b]) * (1 - tol))
        sure[rank == 0] = maybe[rank == 0] = True
        assert maybe[i], (b, i)
        unsure = e[maybe & ~sure].sum() + (tol * e[maybe].sum())
        total = e[maybe].sum()
        at = F(u[b]).astype(np.float64) * total
        lo = e[:i][maybe[:i]].sum()
        assert lo - unsure <= at * (1 + 1e-9) + unsure and at <= lo + e[i] + 2 * unsure, (b, i, lo, at, e[i], unsure)
        assert abs(prob[b] - e[i] / total) <= (e[i] / total) * (unsure / total + 8e-6) + 2.0 ** -30


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("batch,vocab", [(1, 1), (3, 2), (5, 7), (4, 1000), (70, 513), (1, 32000), (200, 4099), (2, 150001)])
def test_against_the_definition(dtype, batch, vocab):
    r = np.random.default_rng(vocab + batch)
    x = torch.from_numpy(r.standard_normal((batch, vocab)) * 2.5).to(DT[dtype])
    for settings in range(3):
        temp = np.where(r.random(batch) < 0.1, 0.0, r.uniform(0.3, 2.0, batch))
        k = np.where(r.random(batch) < 0.4, 0, r.integers(1, max(2, vocab // 3), batch))
        p = np.where(r.random(batch) < 0.4, 1.0, r.uniform(0.05, 1.0, batch))
        m = np.where(r.random(batch) < 0.6, 0.0, r.uniform(0.0, 0.3, batch))
        if settings == 1:
            k[:], p[:], m[:] = 0, 1.0, 0.0            # no filter
        if settings == 2:
            k[:], m[:] = np.minimum(50, vocab), 0.0   # the usual
        u = r.random(batch).astype(F) * F(0.9999999)
        args = (u, temp, k, p, m)
        token, prob = sample(x, *args, strided=3 * (settings == 2))
        check(x, *args, token, prob)
        again = sample(x, *args)
        assert np.array_equal(token, again[0]) and np.array_equal(prob, again[1])


def test_equal_logits_are_drawn_exactly():
    """Equal logits weigh 2^31 each, so every number below is exact: the kept ones are the first by index."""
    V, n = 10007, 64
    r = np.random.default_rng(1)
    for dtype in DT:
        x = torch.full((n, V), 3.5, dtype=DT[dtype])
        u = r.random(n).astype(F) * F(0.9999999)
        k = np.where(np.arange(n) % 2 == 0, 0, r.integers(1, V, n))
        p = np.where(np.arange(n) % 4 < 2, 1.0, r.uniform(0.01, 0.99, n)).astype(F)
        token, prob = sample(x, u, np.full(n, 0.7), k, p, np.zeros(n))
        for b in range(n):
            kept = V if k[b] <= 0 else int(k[b])
            total = kept * 2 ** 31
            kept = sum(1 for _ in range(0)) or int(np.sum(np.arange(kept) * float(2 ** 31) < float(total) * float(p[b])))
            want = int(float(kept * 2 ** 31) * float(u[b])) // 2 ** 31
            assert token[b] == want and prob[b] == F(1.0 / kept), (b, token[b], want)


def test_ties_at_the_cut_go_to_the_lowest_index():
    # 3 large, 1000 equal, the rest far below: top-k cuts into the equal ones
    V = 5000
    for dtype in DT:
        for first in (0, 1777):
            x = torch.full((8, V), -60.0, dtype=DT[dtype])
            x[:, first:first + 1000] = 2.0
            x[:, first + 500:first + 503] = 4.0
            k = np.array([4, 5, 100, 503, 504, 1002, 1003, 2000])
            u = np.full(8, 0.9999999, F)
            token, _ = sample(x, u, np.ones(8), k, np.ones(8), np.zeros(8))
            ties = np.minimum(k - 3, 997)
            order = [i for i in range(first, first + 1000) if not first + 500 <= i < first + 503]
            want = [max(order[t - 1], first + 502) if order[t - 1] > first + 502 else first + 502 for t in ties]
            assert token.tolist() == want


def test_edges_of_the_settings():
    V = 3001
    r = np.random.default_rng(2)
    x = torch.from_numpy(r.standard_normal((16, V)).astype(F))
    best = x.argmax(-1).numpy()
    one = np.ones(16)
    u = np.full(16, 0.999, F)
    cases = {
        "temperature 0": (u, 0 * one, 0 * one, one, 0 * one), "temperature below 0": (u, -one, 0 * one, one, 0 * one),
        "temperature NaN": (u, np.nan * one, 0 * one, one, 0 * one), "top-k 1": (u, one, one, one, 0 * one),
        "top-p 0": (u, one, 0 * one, 0 * one, 0 * one), "top-p tiny": (u, one, 0 * one, 1e-9 * one, 0 * one),
        "min-p 1": (u, one, 0 * one, one, one), "min-p above 1": (u, one, 0 * one, one, 2 * one),
        "tiny temperature": (u, 1e-30 * one, 0 * one, one, 0 * one)}
    for name, args in cases.items():
        token, prob = sample(x, *args)
        assert np.array_equal(token, best) and (prob == 1).all(), name
    # limits that limit nothing
    for args in ((u, one, V * one, one, 0 * one), (u, one, 10 ** 9 * one, 2 * one, -one)):
        token, prob = sample(x, *args)
        want = sample(x, u, one, 0 * one, one, 0 * one)
        assert np.array_equal(token, want[0]) and np.array_equal(prob, want[1])
    # the ends of u: the first kept token, and the last
    x[:] = 0.0
    token, _ = sample(x, np.zeros(16, F), one, 0 * one, one, 0 * one)
    assert (token == 0).all()
    token, _ = sample(x, np.full(16, F(1 - 2.0 ** -24)), one, 0 * one, one, 0 * one)
    assert (token == V - 1).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_masked_and_odd_logits(dtype):
    V, inf = 2000, float("inf")
    x = torch.full((8, V), -inf, dtype=DT[dtype])
    x[1, 1234] = -5.0                                  # one token left
    x[2] = float("nan")
    x[3], x[3, 7] = float("nan"), 1.0
    x[4, 100:104] = inf                                # infinities share
    x[5] = 0.0
    x[5, ::2] = -0.0                                   # zeros of both signs are equal
    x[6, 3], x[6, 9] = 1.0, 0.5
    x[7], x[7, 11] = -30000.0, -29000.0
    u = np.array([0.5, 0.5, 0.5, 0.5, 0.6, 0.25, 0.99, 0.999], F)
    for k, p in ((0, 1.0), (40, 0.99), (1500, 1.0)):
        token, prob = sample(x, u, np.ones(8), np.full(8, k), np.full(8, p), np.zeros(8))
        kept = V if k == 0 else k
        kept = int(np.sum(np.arange(kept) * float(2 ** 31) < float(kept * 2 ** 31) * float(F(p))))
        assert token.tolist() == [-1, 1234, -1, 7, 102, int(kept * 2 ** 31 * float(u[5])) // 2 ** 31, 9, 11]
        assert prob[[0, 2]].tolist() == [0.0, 0.0] and prob[1] == 1 and prob[4] == 0.25


def test_settings_left_out():
    from weight_only_int4_02_gb300 import w4a16
    x = torch.randn(4, 999).cuda()
    u = torch.rand(4).cuda()
    full = w4a16.sample(x, u, torch.ones(4).cuda(), torch.zeros(4, dtype=torch.int32).cuda(), torch.ones(4).cuda(),
                        torch.zeros(4).cuda())
    short = w4a16.sample(x, u)
    assert torch.equal(full[0], short[0]) and torch.equal(full[1], short[1])
    none = w4a16.sample(x[:0], u[:0])
    assert none[0].shape == (0,)


def test_the_same_token_alone_and_in_a_batch():
    from weight_only_int4_02_gb300 import w4a16
    x = (torch.randn(150, 40000) * 3).to(torch.bfloat16).cuda()
    u = torch.rand(150).cuda()
    p = torch.full((150,), 0.9).cuda()
    k = torch.full((150,), 300, dtype=torch.int32).cuda()
    token, prob = w4a16.sample(x, u, top_k=k, top_p=p)
    for b in (0, 77, 149):
        one = w4a16.sample(x[b:b + 1], u[b:b + 1], top_k=k[:1], top_p=p[:1])
        assert one[0][0] == token[b] and one[1][0] == prob[b]
