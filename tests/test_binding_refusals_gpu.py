"""The serving step's Python calls refuse, on the host and before a launch, CUDA tensors that are right but for one property."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(*a, dtype=torch.int32):
    return torch.tensor(a, dtype=dtype, device="cuda")


def every_other(t):
    """t's values, its last dimension's neighbours two elements apart."""
    wide = torch.zeros(t.shape[:-1] + (2 * t.shape[-1],), dtype=t.dtype, device=t.device)
    wide[..., ::2] = t
    return wide[..., ::2]


def refused(call, good, breaks):
    from weight_only_int4_02_gb300 import w4a16
    call(**good)
    torch.cuda.synchronize()
    for name, bad in breaks:
        with pytest.raises(w4a16.W4A16Error) as e:
            call(**dict(good, **{name: bad}))
            pytest.fail("%s was taken: %r" % (name, bad))
        assert e.value.status in (w4a16.ERR_INVALID_ARG, w4a16.ERR_WORKSPACE), name
    torch.cuda.synchronize()
    assert w4a16.check_device_status() == w4a16.OK


def test_tables():
    from weight_only_int4_02_gb300 import w4a16
    seq, new, free = ints(20, 3), ints(2, 3), torch.arange(9, dtype=torch.int32, device="cuda")
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    refused(w4a16.kv4_tables, dict(seq_lens=seq, new_lens=new, free_pages=free, block_table=table, page_size=16, max_tokens=5,
                                   taken=ints(1)),
            [("seq_lens", seq.long()), ("seq_lens", seq[:, None]), ("seq_lens", every_other(seq)), ("seq_lens", seq.cpu()),
             ("seq_lens", [20, 3]), ("new_lens", ints(1, 2, 3)), ("new_lens", new.float()), ("free_pages", free.long()),
             ("free_pages", free[:, None]), ("free_pages", every_other(free)), ("block_table", table.long()),
             ("block_table", table[:1]), ("block_table", table[:1].expand(2, -1)), ("block_table", table.t().contiguous().t()),
             ("block_table", table[0]), ("page_size", 24), ("page_size", 16.0), ("max_tokens", -1), ("max_tokens", 1 << 40),
             ("taken", ints(1, 2)), ("taken", ints(1).long()), ("taken", 0)])


def test_append_and_read():
    from weight_only_int4_02_gb300 import w4a16
    cache = w4a16.kv4_cache(3, 2, 64, 16)
    k = torch.randn(5, 2, 64, device="cuda").to(torch.float16)
    slots = torch.arange(5, device="cuda")
    wide = torch.zeros(5, 2, 72, dtype=torch.float16, device="cuda")
    odd = torch.zeros(5, 2, 68, dtype=torch.float16, device="cuda")
    caches = [("cache", cache.to(torch.int8)), ("cache", cache[:, :, 0]), ("cache", cache.transpose(0, 1).contiguous().transpose(0, 1)),
              ("cache", cache.cpu()), ("page_size", 32), ("page_size", None), ("slots", slots.int()), ("slots", slots[:, None]),
              ("slots", every_other(slots))]
    for name in ("k", "v"):
        caches_and = caches + [(name, k.float()), (name, k.bfloat16()), (name, k[:4]), (name, k[:, :1]), (name, k[:, :1].expand(-1, 2, -1)),
                               (name, k[:1].expand(5, -1, -1)), (name, k[..., :32]), (name, every_other(k)), (name, odd[..., :64]),
                               (name, wide[..., 1:65]), (name, k[0]), (name, k.cpu()), (name, None)]
        refused(w4a16.kv4_append, dict(k=k, v=k, slots=slots, cache=cache, page_size=16), caches_and)
    refused(w4a16.kv4_read, dict(cache=cache, slots=slots, page_size=16, dtype=torch.float32),
            caches + [("dtype", torch.int8), ("dtype", torch.float64)])


def test_attention():
    from weight_only_int4_02_gb300 import w4a16
    cache = w4a16.kv4_cache(3, 2, 64, 16)
    q = torch.randn(3, 4, 64, device="cuda").to(torch.float16)
    table, seq, starts = ints(0, 1, 2, -1).view(2, 2), ints(20, 5), ints(0, 2, 3)
    ws = torch.zeros(w4a16.kv4_workspace_bytes() + 256, dtype=torch.uint8, device="cuda")
    refused(w4a16.kv4_attention, dict(q=q, cache=cache, block_table=table, seq_lens=seq, starts=starts, page_size=16, max_q=2,
                                      scale=0.1, window=0, out=torch.empty_like(q), return_lse=True, workspace=ws),
            [("q", q.float()), ("q", q[:, :3]), ("q", q[..., :32]), ("q", every_other(q)), ("q", q[0]), ("q", q.cpu()),
             ("q", q[:1].expand(3, -1, -1)), ("cache", cache.to(torch.int8)), ("cache", cache[:, :1]), ("page_size", 32),
             ("block_table", table.long()), ("block_table", every_other(table)), ("block_table", table[:1]), ("block_table", table[0]),
             ("block_table", torch.zeros(4, dtype=torch.int32, device="cuda").as_strided((2, 2), (1, 1))),
             ("seq_lens", seq.long()), ("seq_lens", ints(20, 5, 1)), ("seq_lens", every_other(seq)), ("starts", ints(0, 2)),
             ("starts", starts.long()), ("max_q", -1), ("max_q", "2"), ("scale", float("nan")), ("scale", float("inf")),
             ("scale", "0.1"), ("window", -1), ("window", 1.5), ("out", q.bfloat16()), ("out", q[:2].clone()),
             ("out", every_other(q)), ("out", q.cpu()), ("workspace", ws[:1024]), ("workspace", ws[16:]), ("workspace", ws.cpu())])


def test_sample():
    from weight_only_int4_02_gb300 import w4a16
    x, u, one = torch.randn(4, 100, device="cuda"), torch.rand(4, device="cuda"), torch.ones(4, device="cuda")
    refused(w4a16.sample, dict(logits=x, u=u, temperature=one, top_k=ints(1, 2, 3, 0), top_p=one, min_p=one),
            [("logits", x.double()), ("logits", x[0]), ("logits", every_other(x)), ("logits", x[:3]), ("logits", x.cpu()),
             ("logits", x.view(-1).as_strided((4, 100), (50, 1))), ("logits", torch.zeros(4, 262145, device="cuda")),
             ("logits", x[:, :0]), ("u", u.double()), ("u", u[:3]), ("u", every_other(u)), ("u", 0.5), ("temperature", one[:1]),
             ("temperature", one.half()), ("temperature", 0.7), ("top_k", one), ("top_k", ints(1, 2, 3)), ("top_p", one.double()),
             ("top_p", one[:2]), ("min_p", one[:1].expand(4)), ("min_p", one.cpu())])
