"""The example decoder with rotations, norms for each head and a cache of 4 or 8 bits: its steps against plain torch in 64 bits."""
import numpy as np
import pytest

from tests import kv8_reference as ref8, serving_reference as ref4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("qk_norm", [False, True])
def test_a_step_against_plain_torch(bits, qk_norm):
    """What a layer's attention makes of its projections, and what its cache holds after a prompt and a decode step."""
    from weight_only_int4_02_gb300 import serve, w4a16
    model = serve.Decoder(layers=1, ffn=1024, vocab=1024, cache_bits=bits, rope_base=10000.0, qk_norm=qk_norm, max_positions=64)
    layer, page = model.layers[0], 16
    caches = model.caches(8, page)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(8, dtype=torch.int32, device="cuda").flip(0)
    taken, seq = None, torch.zeros(2, dtype=torch.int32, device="cuda")
    rope = model.rope.cpu().numpy()
    held = ref8.append if bits == 8 else None
    want = caches[0].cpu().numpy()
    most = [0.0, 0.0]
    for new in ([23, 4], [1, 1]):
        n = torch.tensor(new, dtype=torch.int32, device="cuda")
        seq = seq + n
        T = sum(new)
        slots, positions, starts, taken = w4a16.kv4_tables(seq, n, free, table, page, T, taken=taken)
        tokens = torch.randint(0, 1024, (T,), device="cuda")
        logits = model.step(tokens, caches, table, seq, slots, starts, page, max(new), positions)
        assert logits.shape == (2, 1024) and torch.isfinite(logits).all()
        qkv = layer["qkv"](serve.rms_norm(model.embedding[tokens])).view(T, 12, 128)
        q, k, v = (x.double().cpu().numpy() for x in qkv.split([8, 2, 2], 1))
        if qk_norm:
            q, k = (x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w.double().cpu().numpy()
                    for x, w in ((q, layer["q_norm"]), (k, layer["k_norm"])))
        pos = positions.cpu().numpy()
        q, k = (ref8.rotate(x, pos, rope, False) for x in (q, k))
        at = slots.cpu().numpy()
        stored_k, stored_v = (w4a16.kv4_read if bits == 4 else w4a16.kv8_read)(caches[0], slots, page, dtype=torch.float32)
        # half a step of what is stored (a step of 4 bits is the row's range over 15, of 8 bits the tile's largest over 127: of the run or
        # of what was there, so of the prompt's too in the decode step: its scale max(old, max|x| / 127) never shrinks, and half of it is
        # up to most / 254, whatever the new tokens' own largest), once more for codes rounded again, and the row's binary16 rounding
        for i, (got, x) in enumerate(((stored_k, k), (stored_v, v))):
            most[i] = max(most[i], np.abs(x).max())
            largest = most[i] if bits == 8 else np.abs(x).max()
            step = 2 * largest / 15 if bits == 4 else largest / 127
            err = np.abs(got.double().cpu().numpy() - x)
            assert (err <= step * (1.1 if bits == 4 else 0.6) + 2.0 ** -10 * largest).all()
        if bits == 8 and not qk_norm:   # keys rotated as they are stored: byte for byte
            turned = ref8.rotate(qkv[:, 8:10].float().cpu().numpy(), pos, rope, False)
            want = held(want, turned, qkv[:, 10:].float().cpu().numpy(), at, page)
            assert np.array_equal(caches[0].cpu().numpy(), want)
        # attention over what the cache holds, from the projections
        again = qkv.clone()
        out = model.attention(layer, again, caches[0], table, seq, slots, starts, page, max(new), positions)
        attend = ref8.attention if bits == 8 else ref4.attention
        o = attend(q, caches[0].cpu().numpy(), table.cpu().numpy(), seq.cpu().numpy(), starts.cpu().numpy(), page, 128 ** -0.5, 0)[0]
        # queries rounded to binary16 move scores of a few units by 2^-11 of them, outputs by as much
        assert np.abs(out.double().cpu().numpy() - o).max() <= 2.0 ** -7 * np.abs(o).max()


def test_requests_together_draw_what_they_draw_alone():
    from weight_only_int4_02_gb300 import serve, w4a16
    model = serve.Decoder(layers=2, ffn=1024, vocab=1024, cache_bits=8, rope_base=10000.0, qk_norm=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompts = [torch.randint(0, 1024, (n,), generator=g, device="cuda") for n in (5, 40, 1, 17)]
    greedy = dict(steps=8, max_len=64, temperature=0.0)
    together = serve.generate(model, prompts, **greedy)
    assert together.shape == (4, 8) and (together >= 0).all() and (together < 1024).all()
    assert torch.equal(together, serve.generate(model, prompts, **greedy))
    for i, p in enumerate(prompts):      # the first token has a margin; a GEMM's sums may depend on the number of rows
        assert serve.generate(model, [p], **greedy)[0, 0] == together[i, 0]
    assert w4a16.check_device_status() == w4a16.OK


@pytest.mark.parametrize("bits", ["4", "8"])
def test_the_command_runs(capsys, monkeypatch, bits):
    from weight_only_int4_02_gb300 import serve
    monkeypatch.setattr("sys.argv", ["serve", "--requests", "3", "--steps", "3", "--layers", "1", "--prompt", "40", "--cache-bits", bits,
                                     "--rope-base", "10000", "--qk-norm"])
    serve.main()
    assert "3 tokens for each of 3 requests" in capsys.readouterr().out


def test_refusals():
    from weight_only_int4_02_gb300 import serve
    with pytest.raises(ValueError):
        serve.Decoder(layers=1, cache_bits=6)
    model = serve.Decoder(layers=1, ffn=1024, vocab=1024, rope_base=10000.0, max_positions=16)
    with pytest.raises(ValueError):
        serve.generate(model, [torch.zeros(12, dtype=torch.int64, device="cuda")], 6, max_len=64)
    with pytest.raises(ValueError):
        model.step(torch.zeros(1, dtype=torch.int64, device="cuda"), None, None, None, None, None, 16, 1)
