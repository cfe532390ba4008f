"""The norms', the rotation's and the 8-bit cache's C ABI and their oracle without a GPU: refusals before any device work,
sizes, the layout and the stored values of the oracle."""
import ctypes

import numpy as np
import pytest

from tests import kv8_reference as ref


@pytest.fixture(scope="module")
def lib():
    from weight_only_int4_02_gb300 import build
    build.build()
    from weight_only_int4_02_gb300 import w4a16
    return w4a16.lib()


@pytest.fixture(scope="module")
def ptr():
    buf = (ctypes.c_uint8 * 256)()
    yield (ctypes.addressof(buf) + 63) // 64 * 64
    del buf


def refuses(call, good, breaks):
    from weight_only_int4_02_gb300 import w4a16 as w
    for bad in breaks:
        args = list(good)
        for i, value in (bad if isinstance(bad[0], tuple) else [bad]):
            args[i] = value
        assert call(*args) == w.ERR_INVALID_ARG, bad


def test_page_bytes(lib):
    assert lib.w4a16_kv8_page_bytes(8, 128, 16) == 8 * (32 * 128 + 16)
    assert lib.w4a16_kv8_page_bytes(1, 64, 256) == 16 * (32 * 64 + 16)
    for heads, dim, page in ((0, 128, 16), (1, 96, 16), (1, 128, 8), (1, 128, 24), (1, 128, 512), (-1, 64, 16)):
        assert lib.w4a16_kv8_page_bytes(heads, dim, page) == 0


def test_rope_table_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    good = [ptr, 4, 64, 10000.0, None]
    refuses(lib.w4a16_rope_table, good, [(0, None), (0, ptr + 8), (1, -1), (2, 0), (2, -8), (2, 12), (3, 0.0), (3, -1.0),
                                         (3, float("nan")), (3, float("inf"))])
    assert lib.w4a16_rope_table(None, 0, 64, 10000.0, None) == w.OK


def test_norm_rope_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr
    #  0  1    2    3  4    5    6  7    8    9  10   11   12 13 14    15 16 17 18   19 20 21 22 23   24 25
    good = [p, 512, 128, p, 512, 128, p, 256, 128, p, 256, 128, p, p, 1e-6, p, p, 9, 128, 0, 2, 4, 2, 128, 0, None]
    refuses(lib.w4a16_qk_norm_rope, good, [
        (0, None), (0, p + 8), (1, 64), (1, 516), (2, 120), (3, None), (3, p + 2), (4, 100), (5, 132), (6, None), (7, 8), (8, 64),
        (9, None), (9, p + 8), (10, 0), (11, -128), (12, p + 2), (13, p + 8), (14, -1.0), (14, float("nan")), (14, float("inf")),
        (15, None), (15, p + 2), (16, None), (16, p + 4), (17, 0), (17, -1), (18, 0), (18, 136), (18, 20), (18, -8), (19, 2),
        (19, -1), (20, -1), (21, -1), (22, -1), (23, 96), (23, 0), (24, 2), (24, -1), ((20, 2 ** 30), (21, 16))])
    for none in (20,):
        assert lib.w4a16_qk_norm_rope(*(good[:none] + [0] + good[none + 1:])) == w.OK
    args = list(good)
    args[21] = args[22] = 0
    assert lib.w4a16_qk_norm_rope(*args) == w.OK


def test_append_and_read_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr
    #       0  1    2    3  4    5    6  7  8  9  10   11 12 13 14 15 16   17  18 19
    good = [p, 256, 128, p, 256, 128, p, p, p, 9, 128, 0, p, 4, 3, 2, 128, 16, 0, None]
    refuses(lib.w4a16_kv8_append, good, [
        (0, None), (0, p + 8), (1, 64), (1, 260), (2, 120), (3, None), (4, 0), (5, 100), (6, None), (6, p + 4), (7, None), (7, p + 2),
        (8, None), (8, p + 8), (9, 0), (10, 0), (10, 136), (10, 4), (11, 2), (12, None), (12, p + 4), (13, -1), (14, -1), (15, 0),
        (16, 80), (17, 20), (18, 2), (18, -1), ((14, 1 << 20), (15, 1 << 12))])
    assert lib.w4a16_kv8_append(*(good[:14] + [0] + good[15:])) == w.OK
    good = [p, 4, p, p, p, 3, 2, 128, 16, 2, None]
    refuses(lib.w4a16_kv8_read, good, [(0, None), (1, -1), (2, None), (3, p + 2), (4, None), (5, -1), (6, 0), (7, 32), (8, 0), (9, 3)])
    assert lib.w4a16_kv8_read(*(good[:5] + [0] + good[6:])) == w.OK


def test_attention_refusals(lib, ptr):
    from weight_only_int4_02_gb300 import w4a16 as w
    p = ptr
    good = [p, 512, 128, p, 4, p, 8, 8, p, p, p, 512, 128, None, 2, 2, 4, 2, 128, 16, 1, 0.1, 0, 0, None, 0, None]
    refuses(lib.w4a16_kv8_attention, good, [
        (0, None), (0, p + 2), (1, 100), (1, 516), (2, 64), (3, None), (3, p + 8), (4, -1), (5, None), (6, 4), (7, -1), (8, None),
        (9, None), (10, None), (10, p + 8), (11, 8), (12, 132), (13, p + 2), (14, -1), (15, -1), (16, 0), (16, 3), (17, 0), (18, 80),
        (19, 17), (20, -1), (21, float("nan")), (21, float("inf")), (22, -1), (23, 2), (24, p + 64)])
    for i in (14, 15):
        assert lib.w4a16_kv8_attention(*(good[:i] + [0] + good[i + 1:])) == w.OK


def test_force_path_takes_its_values(lib):
    assert lib.w4a16_kv8_force_path(2) == 0 and lib.w4a16_kv8_force_path(3) == -1 and lib.w4a16_kv8_force_path(0) == 2


@pytest.mark.parametrize("call", ["qk_norm_rope", "kv8_append", "kv8_read", "kv8_attention"])
def test_the_binding_refuses_wrong_tensors(lib, call):
    torch = pytest.importorskip("torch")
    from weight_only_int4_02_gb300 import w4a16 as w
    cpu = torch.zeros(4, 2, 64, dtype=torch.float16)
    ints = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros((2, 2, 1, 32 * 64 + 16), dtype=torch.uint8)
    with pytest.raises(w.W4A16Error) as e:
        if call == "qk_norm_rope":
            w.qk_norm_rope(cpu, cpu)
        elif call == "kv8_append":
            w.kv8_append(cpu, cpu, ints.long(), cache, 16)
        elif call == "kv8_read":
            w.kv8_read(cache, ints.long(), 16)
        else:
            w.kv8_attention(cpu, cache, ints[:, None], ints, ints, 16, 1)
    assert e.value.status == w.ERR_INVALID_ARG


def test_python_refuses_sizes_that_are_not_there(lib):
    from weight_only_int4_02_gb300 import w4a16 as w
    for call in (lambda: w.kv8_cache(2, 2, 96, 16, device="cpu"), lambda: w.kv8_cache(-1, 2, 64, 16, device="cpu"),
                 lambda: w.rope_table(0, 64), lambda: w.rope_table(4, 0), lambda: w.kv8_force_path(3)):
        with pytest.raises(w.W4A16Error) as e:
            call()
        assert e.value.status == w.ERR_INVALID_ARG
    assert w.kv8_cache(3, 2, 64, 32, device="cpu").shape == (3, 2, 2, 32 * 64 + 16)


@pytest.mark.parametrize("D", [64, 128])
def test_the_oracle_decodes_what_it_encodes(D):
    r = np.random.default_rng(D)
    parts = [r.integers(0, 256, (3, 16, D), dtype=np.uint8), r.integers(0, 256, (3, 16, D), dtype=np.uint8),
             r.random(3).astype(np.float32), r.random(3).astype(np.float32)]
    for a, b in zip(parts, ref.decode(ref.encode(*parts), D)):
        assert np.array_equal(a, b)


def test_the_oracle_stores_to_the_nearest_step():
    """A run is half a step of its scale off, and two roundings in x / s: 127 steps of 2^-23. Codes that are rounded again,
    each time by half a step of the scale as it is then, are off by at most that many halves of the last one."""
    r = np.random.default_rng(0)
    x = (r.standard_normal((16, 64)) * np.exp(0.5 * r.standard_normal((16, 1)))).astype(np.float32)
    code, scale = np.zeros((16, 64), np.uint8), np.float32(7)
    for off in range(16):
        code, scale = ref.store(code, scale, x[off:off + 1], off)
        assert scale == np.abs(x[:off + 1]).max() * (np.float32(1) / np.float32(127))
        value = (code[:off + 1].astype(np.float64) - 128) * float(scale)
        steps = np.abs(value - x[:off + 1]) / float(scale)
        assert (steps[-1] <= 0.5 + 127 * 2.0 ** -23).all() and (steps <= 0.5 * (off + 1) + 0.001).all()
    whole, s = ref.store(np.zeros((16, 64), np.uint8), np.float32(7), x, 0)
    assert s == scale and (np.abs((whole.astype(np.float64) - 128) * float(s) - x) <= float(s) * (0.5 + 127 * 2.0 ** -23)).all()


def test_the_oracle_turns_pairs_by_their_angles():
    """As complex numbers times exp(i p base^(-2i / rot)), both pairings, in 64 bits."""
    r = np.random.default_rng(1)
    x, pos, rot = r.standard_normal((5, 2, 64)), np.array([0, 1, 7, 100, 2999]), 24
    table = ref.rope_table(3000, rot).astype(np.float64)
    turn = np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot))[:, None]
    for interleaved in (False, True):
        z = x[..., 0:rot:2] + 1j * x[..., 1:rot:2] if interleaved else x[..., :rot // 2] + 1j * x[..., rot // 2:rot]
        y = ref.rotate(x, pos, table, interleaved)
        got = y[..., 0:rot:2] + 1j * y[..., 1:rot:2] if interleaved else y[..., :rot // 2] + 1j * y[..., rot // 2:rot]
        assert np.abs(got - z * turn).max() < 1e-6 and np.array_equal(y[..., rot:], x[..., rot:])


def test_append_refuses_heads_past_its_grid(lib, ptr):
    """Two CTAs and more take a head of a window of the list: 2^30 heads of a few tokens are 2^31 of them."""
    p = ptr
    good = [p, 256, 128, p, 256, 128, p, p, p, 9, 128, 0, p, 4, 1, 2, 128, 16, 0, None]
    refuses(lib.w4a16_kv8_append, good, [(15, (1 << 29) + 1), (15, 1 << 30), (15, (1 << 31) - 300)])


def test_norms_refuse_heads_whose_last_pass_overflows(lib, ptr):
    """A warp takes up to 64 heads: where the last warp begins less than that below 2^31, the head behind its rows has no number."""
    p = ptr
    good = [p, 512, 128, p, 512, 128, p, 256, 128, p, 256, 128, p, p, 1e-6, p, p, 9, 128, 0, 1, 4, 2, 128, 0, None]
    refuses(lib.w4a16_qk_norm_rope, good, [(21, (1 << 31) - 30), ((21, 0), (22, (1 << 31) - 30)), ((21, 0), (22, (1 << 31) - 60), (23, 64))])


def test_rotation_tables_past_32_bits_are_refused():
    """Rows that the C call would count as 4 or 0: refused before any memory is taken (there is no such device here either)."""
    from weight_only_int4_02_gb300 import w4a16 as w
    for rows, rot in (((1 << 32) + 4, 64), (1 << 32, 64), (1 << 31, 8), (4, (1 << 32) + 64), (4, 65544)):
        with pytest.raises(w.W4A16Error):
            w.rope_table(rows, rot)
