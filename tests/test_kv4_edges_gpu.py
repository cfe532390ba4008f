"""The 4-bit key-value cache's calls at the ends of their arguments' ranges, against their definitions."""
import numpy as np
import pytest

from tests import serving_reference as ref

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
