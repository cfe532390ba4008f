"""Attention where scores are so large that their FP32 spacing is no longer small beside one: a softmax that measures scores from
a reference has to round both alike, or the key that wins gets a weight far from one (past the range of the number that it is fed as,
or nothing).

One key of each head lies along the queries, so that it wins by most of its score and the definition gives its value row: every
other weight is exp(-1000) or less. Tolerances: the value row through the MMAs, as in the caches' own tests, 2^-20 of the bare
codes' mass, at most four times the largest value, half a step for the output and, where the tcgen05 kernel feeds bfloat16 outputs' weights as
one binary16 number, 2^-11 of the value. The log-sum is the winner's score: sums of head_dim products of q and bare codes,
16 * 2^-24 of their mass, which is at most three times the score here, and its conversions, 2^-22."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def compare(bits, path, nq, dtype, k, v, q, powers, scales, least=1000, window=0):
    """Attention of the last nq tokens over keys and values [seq][heads][D], for queries q [nq][2 heads * group][D] of several
    sizes. Keys that are not the largest lie `least` below it; those that are equal share."""
    from weight_only_int4_02_gb300 import w4a16
    append, read, attention, force = ((w4a16.kv4_append, w4a16.kv4_read, w4a16.kv4_attention, w4a16.kv4_force_path) if bits == 4 else
                                      (w4a16.kv8_append, w4a16.kv8_read, w4a16.kv8_attention, w4a16.kv8_force_path))
    page, (seq, heads, D), t = 16, k.shape, getattr(torch, dtype)
    pages, group, half = -(-seq // page), q.shape[1] // heads, dtype == "float16"
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    cache = (w4a16.kv4_cache if bits == 4 else w4a16.kv8_cache)(pages, heads, D, page)
    slots = torch.arange(seq, device="cuda")
    append(k.to(t).cuda(), v.to(t).cuda(), slots, cache, page)
    key, val = (x.double().cpu() for x in read(cache, slots, page, dtype=torch.float32))
    lens, starts = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([seq], [0, nq]))
    before = force(path)
    try:
        for power in powers:
            for scale in scales if power < 110 else (1.0,):
                x = (q * (2.0 ** power if scale > 0 else -2.0 ** power)).to(t)
                out, lse = attention(x.cuda(), cache, table, lens, starts, page, nq, scale=scale, window=window, return_lse=True)
                s = torch.einsum("thgd,khd->thgk", x.double().view(nq, heads, group, D), key) * scale
                at, pos = torch.arange(seq), torch.arange(seq - nq, seq).view(-1, 1, 1, 1)
                s = s.masked_fill((at > pos) | (at <= pos - (window or seq)), -np.inf)
                top = s.amax(-1, keepdim=True)
                equal = s >= top * (1 - 1e-12)
                assert (equal | (s < top - least)).all()
                p = equal.double() / equal.sum(-1, keepdim=True)
                want = torch.einsum("thgk,khd->thgd", p, val).reshape(out.shape)
                bound = (2.0 ** -11 if half else 2.0 ** -8) * 1.01 * want.abs() + 2.0 ** -20 * val.abs().amax() * 4
                if path == 2 and not half:
                    bound = bound + 2.0 ** -11 * torch.einsum("thgk,khd->thgd", p, val.abs()).reshape(out.shape)
                err = (out.double().cpu() - want).abs()
                assert bool((err <= bound).all()), (power, scale, float((err / bound).max()))
                log = (top[..., 0] + equal.sum(-1).log()).view(nq, -1)
                assert bool(((lse.double().cpu() - log).abs() <= (2 * 16 * 3 * 2.0 ** -24 + 2.0 ** -22) * log.abs()).all()), (power, scale)
    finally:
        force(before)
    assert w4a16.check_device_status() == w4a16.OK


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("path,nq", [(1, 1), (1, 6), (2, 40)])
@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("winner", [0, 100, 159])
def test_the_largest_score_takes_all(bits, path, nq, D, dtype, winner):
    heads, group, seq = 2, 4, 200
    g = torch.Generator().manual_seed(winner + nq)
    along = torch.randn(heads, D, generator=g).sign()                       # each head's direction
    k, v = 0.25 * torch.randn(seq, heads, D, generator=g), torch.randn(seq, heads, D, generator=g)
    k[winner] = along
    q = (along.repeat_interleave(group, 0) * (1 + 0.25 * torch.rand(nq, heads * group, D, generator=g))).double()
    compare(bits, path, nq, dtype, k, v, q, (6, 14) if dtype == "float16" else (6, 20, 26, 30, 60, 110), (1.0, 17.3, -17.3))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("path,nq", [(1, 3), (2, 40)])
@pytest.mark.parametrize("D,dtype", [(64, "float16"), (128, "bfloat16")])
@pytest.mark.parametrize("order", ["up", "down", "both"])
def test_scores_that_pass_the_far_ones_step_by_step(bits, path, nq, D, dtype, order):
    """From 2^18 to 2^21 and more in powers of two, a new largest one in every few tokens on the way up: keys of a head lie all along one
    direction, in steps of an eighth that no rounding of theirs joins."""
    heads, group, seq = 2, 4, 640
    g = torch.Generator().manual_seed(seq + nq)
    along = torch.randn(heads, D, generator=g).sign()
    step = torch.arange(seq) // 32 % 20
    size = 0.875 ** {"up": 19 - step, "down": step, "both": (step * 2 - 19).abs()}[order]
    k, v = along * size.view(-1, 1, 1), torch.randn(seq, heads, D, generator=g)
    q = along.repeat_interleave(group, 0).expand(nq, -1, -1).double()
    compare(bits, path, nq, dtype, k, v, q, (8, 12, 14) if dtype == "float16" else (8, 12, 14, 18, 40), (1.0, 17.3, -17.3))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("path,nq", [(1, 2), (2, 70)])
@pytest.mark.parametrize("D,dtype", [(64, "bfloat16"), (128, "float16")])
@pytest.mark.parametrize("window", [0, 777])
def test_far_scores_in_the_parts_of_a_long_request(bits, path, nq, D, dtype, window):
    """Parts whose references lie far apart are joined, some of them with nothing but small scores; a window's edge moves with the query."""
    heads, group, seq = 1, 3, 3100
    g = torch.Generator().manual_seed(seq)
    along = torch.randn(heads, D, generator=g).sign()
    step = torch.randint(0, 20, (seq // 50 + 1,), generator=g).repeat_interleave(50)[:seq]
    k, v = along * (0.875 ** step).view(-1, 1, 1), torch.randn(seq, heads, D, generator=g) * torch.exp(torch.randn(seq, 1, 1, generator=g))
    q = along.repeat_interleave(group, 0).expand(nq, -1, -1).double()
    compare(bits, path, nq, dtype, k, v, q, (12, 14) if dtype == "float16" else (12, 18, 40), (1.0, -17.3), least=100, window=window)
