"""What the Python calls make of their arguments' strides, streams and flags."""
import numpy as np
import pytest

from tests.test_kv4_gpu import batch_of, cuda

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,batch", [(1, 5), (999, 8), (40000, 200)])
def test_several_draws_from_one_row_of_logits(dtype, vocab, batch):
    from weight_only_int4_02_gb300 import w4a16
    x = (torch.randn(1, vocab, device="cuda") * 3).to(dtype)
    u = torch.rand(batch, device="cuda")
    p = torch.full((batch,), 0.9, device="cuda")
    for rows in (x.expand(batch, -1), x[0].expand(batch, -1)):
        assert rows.stride(0) == 0
        got, want = w4a16.sample(rows, u, top_p=p), w4a16.sample(rows.contiguous(), u, top_p=p)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("nq", [1, 3, 40])
def test_requests_over_one_row_of_the_block_table(nq):
    """Several requests that share a prompt's pages: stride 0 between the table's rows."""
    from weight_only_int4_02_gb300 import w4a16
    n = 5
    q, cache, table, seq, starts = batch_of([300], [nq], 2, 4, 64, 16, "bfloat16", 3)
    q = (torch.randn(n * nq, 8, 64) * 0.5).to(q.dtype).cuda()
    seq = cuda(np.array([300, 41, 299, 160, 0], np.int32))
    starts = cuda(np.arange(0, n * nq + 1, nq, dtype=np.int32))
    rows = cuda(table).expand(n, -1)
    assert rows.stride(0) == 0
    for path in (0, 2):
        before = w4a16.kv4_force_path(path)
        try:
            got = w4a16.kv4_attention(q, cuda(cache), rows, seq, starts, 16, nq, return_lse=True)
            want = w4a16.kv4_attention(q, cuda(cache), rows.contiguous(), seq, starts, 16, nq, return_lse=True)
        finally:
            w4a16.kv4_force_path(before)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_that_overlap_are_refused():
    """A stride below a row's length, other than 0, reaches the library as it is and is refused there."""
    from weight_only_int4_02_gb300 import w4a16
    x = torch.zeros(64, device="cuda").as_strided((4, 16), (8, 1))
    with pytest.raises(w4a16.W4A16Error):
        w4a16.sample(x, torch.zeros(4, device="cuda"))
    assert w4a16.sample(x[:1], torch.zeros(1, device="cuda"))[0].tolist() == [0]   # a single row's stride is never used
    q, cache, table, seq, starts = batch_of([90, 70], [1, 1], 1, 2, 64, 16, "float16", 1)
    rows = torch.zeros(64, dtype=torch.int32, device="cuda").as_strided((2, 7), (5, 1))
    with pytest.raises(w4a16.W4A16Error):
        w4a16.kv4_attention(q.cuda(), cuda(cache), rows, cuda(seq), cuda(starts), 16, 1)


def stream_of(t):
    """The stream whose pool a tensor's memory belongs to."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def test_outputs_belong_to_the_stream_of_the_call():
    """As under torch.cuda.stream(s): memory that the current stream may still use is not handed out."""
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([90, 30], [1, 1], 2, 2, 64, 16, "float16", 1)
    q, cache, table, seq, starts = q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts)
    x, u = torch.randn(2, 1000, device="cuda"), torch.rand(2, device="cuda")
    free = torch.arange(64, dtype=torch.int32, device="cuda")
    slots, new, rows = torch.arange(16, device="cuda"), ints(1, 1), table.clone()
    calls = (lambda **k: w4a16.kv4_tables(seq, new, free, rows, 16, 2, **k),   # the same rows again and again
             lambda **k: w4a16.kv4_read(cache, slots, 16, **k),
             lambda **k: w4a16.kv4_attention(q, cache, table, seq, starts, 16, 1, return_lse=True, **k),
             lambda **k: w4a16.sample(x, u, **k))
    s = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = call(stream=s)
        s.synchronize()
        for a, b in zip(got, want):
            assert stream_of(a) == s.cuda_stream and stream_of(b) == torch.cuda.current_stream().cuda_stream
            assert torch.equal(a, b)
        assert torch.cuda.current_stream().cuda_stream == torch.cuda.default_stream().cuda_stream


def test_the_matmuls_outputs_belong_to_the_stream_of_the_call():
    from weight_only_int4_02_gb300 import w4a16
    K, N, G = 256, 512, 128
    codes = torch.randint(0, 16, (K, N), dtype=torch.uint8, device="cuda")
    codes.view(K // 4, 4, N)[:, 2:] = 8              # two of every four: also 2:4 sparse
    scales = torch.rand(K // G, N, device="cuda").to(torch.float16)
    zeros = torch.randint(0, 16, (K // G, N), dtype=torch.uint8, device="cuda")
    x = torch.randn(4, K, device="cuda").to(torch.float16)
    xb = x.bfloat16()
    w, zp = w4a16.pack(codes, scales, G), w4a16.pack_zeros(zeros, K, G)
    wb, w8, ws = w4a16.pack(codes, scales.bfloat16(), G), w4a16.w8_pack(codes, scales, G), w4a16.sp_pack(codes, scales, G)
    space = torch.zeros(w4a16.workspace_bytes(4, N, K, G), dtype=torch.uint8, device="cuda")
    calls = (lambda **k: w4a16.pack(codes, scales, G, **k), lambda **k: w4a16.pack_zeros(zeros, K, G, **k),
             lambda **k: w4a16.w8_pack(codes, scales, G, **k), lambda **k: w4a16.sp_pack(codes, scales, G, **k),
             lambda **k: w4a16.gemm(x, *w, N, G, **k), lambda **k: w4a16.gemm_ws(x, *w, N, G, space, **k),
             lambda **k: w4a16.gemm_noalloc(x, *w, N, G, **k), lambda **k: w4a16.gemm_fused(x, *w, N, G, **k),
             lambda **k: w4a16.gemm_strided(x, *w, N, G, **k), lambda **k: w4a16.gemm_zp(x, *w, zp, N, G, **k),
             lambda **k: w4a16.w8_gemm(x, *w8, N, G, **k), lambda **k: w4a16.bf16_gemm(xb, *wb, N, G, **k),
             lambda **k: w4a16.sp_gemm(x, *ws, N, G, **k))
    s = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = call(stream=s)
        s.synchronize()
        for a, b in zip(got, want) if isinstance(got, tuple) else ((got, want),):
            assert stream_of(a) == s.cuda_stream and stream_of(b) == torch.cuda.current_stream().cuda_stream
            assert torch.equal(a, b)
    assert w4a16.check_device_status() == w4a16.OK


@pytest.mark.parametrize("flag", [True, 1, np.bool_(True)])
def test_any_true_value_asks_for_the_log_sums(flag):
    from weight_only_int4_02_gb300 import w4a16
    q, cache, table, seq, starts = batch_of([90], [1], 2, 2, 64, 16, "float16", 1)
    args = (q.cuda(), cuda(cache), cuda(table), cuda(seq), cuda(starts), 16, 1)
    out, lse = w4a16.kv4_attention(*args, return_lse=flag)
    assert lse.shape == (1, 4) and torch.isfinite(lse).all()
    assert torch.equal(out, w4a16.kv4_attention(*args, return_lse=type(flag)(0)))
