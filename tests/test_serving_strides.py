"""The C ABI's rule for rows that are only read: a stride of 0 or of at least a row's length (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from weight_only_int4_02_gb300 import build
    build.build()
    from weight_only_int4_02_gb300 import w4a16
    return w4a16.lib()


@pytest.fixture(scope="module")
def at():
    buf = (ctypes.c_uint8 * 256)()
    yield (ctypes.addressof(buf) + 63) // 64 * 64
    del buf


@pytest.mark.parametrize("stride,fine", [(0, True), (100, True), (101, True), (99, False), (1, False), (-1, False), (-100, False)])
def test_row_strides(lib, at, stride, fine):
    """Without a GPU a call whose arguments are right fails later, with another status."""
    import torch
    from weight_only_int4_02_gb300 import w4a16 as w
    if torch.cuda.is_available():
        pytest.skip("would launch on host pointers")
    refused = lib.w4a16_sample(at, stride, at, None, None, None, None, at, None, 2, 100, 0, None) == w.ERR_INVALID_ARG
    assert refused != fine
    refused = lib.w4a16_kv4_attention(at, 512, 128, at, 4, at, stride, 100, at, at, at, 512, 128, None, 2, 2, 4, 2, 128, 16, 1,
                                      0.1, 0, 0, None, 0, None) == w.ERR_INVALID_ARG
    assert refused != fine
