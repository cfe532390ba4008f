"""The serving step's C ABI and its oracle without a GPU: refusals before any device work, sizes,
and the cache layout of the oracle."""
import ctypes

import numpy as np
import pytest

from tests import serving_reference as ref


@pytest.fixture(scope="module")
def lib():
    from weight_only_int4_02_gb300 import build
    build.build()
    from weight_only_int4_02_gb300 import w4a16
    return w4a16.lib()


@pytest.fixture(scope="module")
def ptr():
    buf = (ctypes.c_uint8 * 256)()
    at = (ctypes.addressof(buf) + 63) // 64 * 64
    return buf, at


def test_page_bytes(lib):
    assert lib.w4a16_kv4_page_bytes(8, 128, 16) == 8 * 16 * 134
    assert lib.w4a16_kv4_page_bytes(1, 64, 256) == 256 * 70
    for heads, dim, page in ((0, 128, 16), (1, 96, 16), (1, 128, 8), (1, 128, 24), (1, 128, 512), (-1, 64, 16)):
        assert lib.w4a16_kv4_page_bytes(heads, dim, page) == 0


def test_tables_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr[1]
    good = [p, p, 2, p, 4, p, p + 4, p, 8, 16, p, p, 4, p, None]
    for i, bad in ((2, -1), (4, -1), (8, 0), (9, 0), (9, 48), (12, -1), (0, None), (1, None), (3, None), (6, None),
                   (5, p + 4), (7, None), (10, None), (11, None), (13, None), (0, p + 2), (10, p + 4)):
        args = list(good)
        args[i] = bad
        assert lib.w4a16_kv4_tables(*args) == w.ERR_INVALID_ARG, (i, bad)


def test_append_and_read_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr[1]
    good = [p, 256, 128, p, 256, 128, p, p, 4, 3, 2, 128, 16, 0, None]
    for i, bad in ((0, None), (0, p + 8), (1, 64), (1, 260), (2, 120), (3, None), (4, 0), (5, 100), (6, None), (6, p + 4),
                   (7, None), (7, p + 4), (8, -1), (9, -1), (10, 0), (11, 80), (12, 20), (13, 2), (13, -1)):
        args = list(good)
        args[i] = bad
        assert lib.w4a16_kv4_append(*args) == w.ERR_INVALID_ARG, (i, bad)
    args = list(good)
    args[9], args[10] = 1 << 20, 1 << 12                # rows past 31 bits
    assert lib.w4a16_kv4_append(*args) == w.ERR_INVALID_ARG
    assert lib.w4a16_kv4_append(*(good[:9] + [0] + good[10:])) == w.OK
    good = [p, 4, p, p, p, 3, 2, 128, 16, 2, None]
    for i, bad in ((0, None), (1, -1), (2, None), (3, p + 2), (4, None), (5, -1), (6, 0), (7, 32), (8, 0), (9, 3)):
        args = list(good)
        args[i] = bad
        assert lib.w4a16_kv4_read(*args) == w.ERR_INVALID_ARG, (i, bad)
    assert lib.w4a16_kv4_read(*(good[:5] + [0] + good[6:])) == w.OK


def test_attention_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr[1]
    #        q  qt   qh   cache pages table stride cols seq starts out ot oh  lse batch tokens H kv D page max_q scale win dt ws n s
    good = [p, 512, 128, p, 4, p, 8, 8, p, p, p, 512, 128, None, 2, 2, 4, 2, 128, 16, 1, 0.1, 0, 0, None, 0, None]
    for i, bad in ((0, None), (0, p + 2), (1, 100), (1, 516), (2, 64), (3, None), (3, p + 8), (4, -1), (5, None), (6, 4),
                   (7, -1), (8, None), (9, None), (10, None), (10, p + 8), (11, 8), (12, 132), (13, p + 2), (14, -1),
                   (15, -1), (16, 0), (16, 3), (17, 0), (18, 80), (19, 17), (20, -1), (21, float("nan")),
                   (21, float("inf")), (22, -1), (23, 2), (24, p + 64)):
        args = list(good)
        args[i] = bad
        assert lib.w4a16_kv4_attention(*args) == w.ERR_INVALID_ARG, (i, bad)
    for i in (14, 15):                                   # an empty batch is nothing to do
        args = list(good)
        args[i] = 0
        assert lib.w4a16_kv4_attention(*args) == w.OK


def test_force_path_takes_its_values(lib):
    assert lib.w4a16_kv4_force_path(2) == 0 and lib.w4a16_kv4_force_path(3) == -1 and lib.w4a16_kv4_force_path(0) == 2


def test_sample_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr[1]
    good = [p, 100, p, p, p, p, p, p, p, 2, 100, 0, None]
    for i, bad in ((0, None), (0, p + 1), (1, 99), (2, None), (2, p + 2), (3, p + 1), (4, p + 2), (5, p + 2), (6, p + 2),
                   (7, None), (7, p + 2), (8, p + 2), (9, -1), (9, 1 << 28), (10, 0), (10, 262145), (11, 3), (11, -1)):
        args = list(good)
        args[i] = bad
        assert lib.w4a16_sample(*args) == w.ERR_INVALID_ARG, (i, bad)
    assert lib.w4a16_sample(*(good[:9] + [0] + good[10:])) == w.OK
    args = list(good)
    args[0], args[11] = p + 2, 2                         # FP32 logits on a 2-byte boundary
    assert lib.w4a16_sample(*args) == w.ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["kv4_append", "kv4_attention", "sample", "kv4_tables"])
def test_the_binding_refuses_wrong_tensors(lib, call):
    torch = pytest.importorskip("torch")
    from weight_only_int4_02_gb300 import w4a16 as w
    cpu = torch.zeros(4, 2, 64)
    ints = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros((2, 2, 1, 16 * 70), dtype=torch.uint8)
    with pytest.raises(w.W4A16Error) as e:
        if call == "kv4_append":
            w.kv4_append(cpu, cpu, ints, cache, 16)
        elif call == "kv4_attention":
            w.kv4_attention(cpu, cache, ints[:, None], ints, ints, 16, 1)
        elif call == "sample":
            w.sample(torch.zeros(4, 9, dtype=torch.float64), torch.zeros(4))
        else:
            w.kv4_tables(ints, ints, ints.long(), ints[:, None], 16, 4)
    assert e.value.status == w.ERR_INVALID_ARG


@pytest.mark.parametrize("D,P", [(64, 16), (128, 48)])
def test_the_oracle_decodes_what_it_encodes(D, P):
    r = np.random.default_rng(D)
    parts = [r.integers(0, 16, (P, D)).astype(np.uint8), r.random(P).astype(np.float16), r.integers(0, 16, P).astype(np.uint8),
             r.integers(0, 16, (P, D)).astype(np.uint8), r.random(P).astype(np.float16), r.integers(0, 16, P).astype(np.uint8)]
    for a, b in zip(parts, ref.decode(ref.encode(*parts), D)):
        assert np.array_equal(a, b)


def test_the_oracle_quantises_to_the_nearest_step():
    r = np.random.default_rng(0)
    x = r.standard_normal((200, 64)).astype(np.float32) * np.exp(r.standard_normal((200, 1))).astype(np.float32)
    code, scale, zero = ref.quantise(x)
    value = (code.astype(np.float64) - zero[:, None]) * scale.astype(np.float64)[:, None]
    # half a step, and what rounding the scale to 11 bits (15 steps of 2^-11) and the zero-point (half a step) move
    assert (np.abs(value - x) <= scale.astype(np.float64)[:, None] * (1.0 + 15 * 2.0 ** -11)).all()
    code, scale, zero = ref.quantise(np.array([[0.0] * 64, [np.inf] + [1.0] * 63], np.float32))
    assert scale[0] == 0 and np.isnan(scale[1]) and not code.any() and not zero.any()
