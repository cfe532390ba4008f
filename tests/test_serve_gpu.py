"""The example decoder: its steps against plain torch in 64 bits, and batched against one by one."""
import numpy as np
import pytest

from tests import serving_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_requests_together_draw_what_they_draw_alone():
    from weight_only_int4_02_gb300 import serve, w4a16
    model = serve.Decoder(layers=2, ffn=1024, vocab=1024)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompts = [torch.randint(0, 1024, (n,), generator=g, device="cuda") for n in (5, 40, 1, 17)]
    greedy = dict(steps=8, max_len=64, temperature=0.0)
    together = serve.generate(model, prompts, **greedy)
    assert together.shape == (4, 8) and (together >= 0).all() and (together < 1024).all()
    assert torch.equal(together, serve.generate(model, prompts, **greedy))
    # a GEMM's split of its sums may depend on the number of rows, so a greedy choice could differ where two
    # logits are a rounding apart: the first token of every request, which has a margin, is compared
    for i, p in enumerate(prompts):
        alone = serve.generate(model, [p], **greedy)
        assert alone[0, 0] == together[i, 0]
    assert w4a16.check_device_status() == w4a16.OK


def test_a_step_against_plain_torch():
    """One layer's attention output recomputed in 64 bits from the step's own projections and the
    quantised rows, and the cache's contents after a prompt and a decode step."""
    from weight_only_int4_02_gb300 import serve, w4a16
    from tests.test_kv4_gpu import check
    model = serve.Decoder(layers=1, ffn=1024, vocab=1024)
    page, lens = 16, [23, 4]
    caches = model.caches(8, page)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(8, dtype=torch.int32, device="cuda").flip(0)
    taken, seq = None, torch.zeros(2, dtype=torch.int32, device="cuda")
    kept_k = [[], []]
    for new in (lens, [1, 1]):
        n = torch.tensor(new, dtype=torch.int32, device="cuda")
        seq = seq + n
        T = sum(new)
        tokens = torch.randint(0, 1024, (T,), device="cuda")
        slots, positions, starts, taken = w4a16.kv4_tables(seq, n, free, table, page, T, taken=taken)
        logits = model.step(tokens, caches, table, seq, slots, starts, page, max(new))
        assert logits.shape == (2, 1024) and torch.isfinite(logits).all()
        x = serve.rms_norm(model.embedding[tokens])
        qkv = model.layers[0]["qkv"](x).view(T, 12, 128)
        out, lse = w4a16.kv4_attention(qkv[:, :8], caches[0], table, seq, starts, page, max(new), return_lse=True)
        check(qkv[:, :8].cpu(), caches[0].cpu().numpy(), table.cpu().numpy(), seq.cpu().numpy(), starts.cpu().numpy(),
              page, 0, out, lse)
        for b in range(2):
            kept_k[b].append(qkv[starts[b]:starts[b + 1], 8:10].float().cpu().numpy())
    for b in range(2):
        k = np.concatenate(kept_k[b])
        code, scale, zero = ref.quantise(k)
        want = (code.astype(np.float32) - zero[..., None]) * scale.astype(np.float32)[..., None]
        pos = torch.arange(len(k), device="cuda")
        slot = table[b, pos // page].long() * page + pos % page
        got, _ = w4a16.kv4_read(caches[0], slot, page, dtype=torch.float32)
        assert np.array_equal(got.cpu().numpy(), want)


def test_the_command_runs(capsys, monkeypatch):
    from weight_only_int4_02_gb300 import serve
    monkeypatch.setattr("sys.argv", ["serve", "--requests", "3", "--steps", "3", "--layers", "1", "--prompt", "40"])
    serve.main()
    assert "3 tokens for each of 3 requests" in capsys.readouterr().out
