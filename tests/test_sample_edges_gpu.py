"""Sampling at the ends of the temperature's range: infinite, where all tokens weigh the same, and low,
where few weigh anything."""
import numpy as np
import pytest

from tests.test_sample_gpu import DT, F, check, sample

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("vocab,live", [(7, 7), (1000, 1000), (2048, 2048), (32000, 300), (10007, 10007)])
@pytest.mark.parametrize("temperature", [np.inf, 3.0e38])
def test_an_infinite_temperature_weighs_all_tokens_alike(dtype, vocab, live, temperature):
    """Every finite logit weighs 2^31, so the draw is known exactly: the kept ones are the first by rank."""
    r = np.random.default_rng(vocab)
    n = 12
    x = torch.full((n, vocab), -np.inf, dtype=DT[dtype])
    for b in range(n):
        at = torch.from_numpy(r.permutation(vocab)[:live])
        x[b, at] = torch.from_numpy(r.standard_normal(live) * 3).to(DT[dtype])
    u = r.random(n).astype(F) * F(0.9999999)
    p = np.where(np.arange(n) % 3 == 2, 1.0, r.uniform(0.01, 0.99, n)).astype(F)
    k = np.where(np.arange(n) % 4 == 3, r.integers(1, vocab, n), 0)
    m = np.where(np.arange(n) % 5 == 4, 0.5, 0.0)
    token, prob = sample(x, u, np.full(n, temperature), k, p, m)
    for b in range(n):
        row = x[b].double().numpy()
        order = np.argsort(-row, kind="stable")
        kept = min(live, int(k[b])) if k[b] > 0 else live
        kept = int(np.sum(np.arange(kept) * float(2 ** 31) < float(kept * 2 ** 31) * float(p[b])))
        want = np.sort(order[:kept])[int(float(kept * 2 ** 31) * float(u[b])) // 2 ** 31]
        assert token[b] == want and prob[b] == F(1.0 / kept), (b, token[b], want)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("batch,vocab", [(1, 32000), (3, 131072), (40, 4099)])
@pytest.mark.parametrize("temperature", [0.01, 0.1, 0.2])
def test_low_temperatures(dtype, batch, vocab, temperature):
    r = np.random.default_rng(vocab + batch)
    x = torch.from_numpy(r.standard_normal((batch, vocab)) * 2.5).to(DT[dtype])
    u = r.random(batch).astype(F) * F(0.9999999)
    one = np.ones(batch)
    for k, p, m in ((50, 1.0, 0.0), (50, 0.95, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.02), (0, 1.0, 0.0), (1500, 0.9, 0.0)):
        args = (u, temperature * one, k * one, p * one, m * one)
        check(x, *args, *sample(x, *args))


@pytest.mark.parametrize("batch,vocab", [(700, 300), (1500, 4099), (16384, 70), (20000, 70)])
def test_batches_of_many_rows(batch, vocab):
    """Rows are taken in order of their work, by one of two ways or not at all as the batch is large; each gives what it
    gives in a small batch."""
    r = np.random.default_rng(batch)
    x = torch.from_numpy(r.standard_normal((batch, vocab)) * 3).to(torch.bfloat16)
    args = (r.random(batch).astype(F) * F(0.9999999), np.where(r.random(batch) < 0.2, 0.0, r.uniform(0.3, 2.0, batch)),
            np.where(r.random(batch) < 0.5, 0, r.integers(1, vocab, batch)), np.where(r.random(batch) < 0.5, 1.0, r.uniform(0.05, 1.0, batch)),
            np.where(r.random(batch) < 0.5, 0.0, 0.1))
    token, prob = sample(x, *args)
    some = np.unique(np.concatenate([[0, batch - 1], r.integers(0, batch, 60)]))
    few = sample(x[some], *[a[some] for a in args])
    assert np.array_equal(token[some], few[0]) and np.array_equal(prob[some], few[1])
    check(x[:200], *[a[:200] for a in args], token[:200], prob[:200])
    assert (token >= 0).all() and (token < vocab).all() and (prob > 0).all()
