"""The norms', the rotation's and the 8-bit cache's calls where programs put them together: a decode step in a graph, two streams at
once, lists that come back to a tile, offsets past 32 bits, many heads to one cache."""
import numpy as np
import pytest

from tests import kv8_reference as ref
from tests.test_kv8_gpu import batch_of, cuda, run_and_check, same_cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_a_decode_step_in_a_graph():
    """Captured once, replayed token by token across tiles and pages, against the same calls one by one on another cache."""
    from weight_only_int4_02_gb300 import w4a16
    n, heads, group, D, page, steps = 5, 2, 4, 64, 16, 40
    rope = w4a16.rope_table(200, D)
    prompt = torch.tensor([1, 17, 33, 16, 90], dtype=torch.int32, device="cuda")
    qkv = torch.randn(steps + 1, int(prompt.sum()), heads * (group + 2), D, device="cuda").to(torch.bfloat16)
    weight = (1 + 0.1 * torch.randn(D, device="cuda")).to(torch.bfloat16)

    class State:
        def __init__(self):
            self.cache = w4a16.kv8_cache(80, heads, D, page)
            self.table = torch.full((n, 12), -1, dtype=torch.int32, device="cuda")
            self.free = torch.arange(80, dtype=torch.int32, device="cuda").flip(0)
            self.taken = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.seq = torch.zeros(n, dtype=torch.int32, device="cuda")

        def step(self, x, new, tokens, max_q):
            self.seq += new
            slots, positions, starts, taken = w4a16.kv4_tables(self.seq, new, self.free, self.table, page, tokens, taken=self.taken)
            self.taken.copy_(taken)
            q, k, v = x.split([heads * group, heads, heads], 1)
            q, k = w4a16.qk_norm_rope(q, k, positions, rope, q_weight=weight, k_weight=weight)
            w4a16.kv8_append(k, v, slots, self.cache, page)
            return w4a16.kv8_attention(q, self.cache, self.table, self.seq, starts, page, max_q)

    one = torch.ones_like(prompt)
    eager, replayed = State(), State()
    for s in (eager, replayed):
        s.step(qkv[0].clone(), prompt, qkv.shape[1], 90)
    x = torch.zeros(n, heads * (group + 2), D, dtype=torch.bfloat16, device="cuda")
    before = [t.clone() for t in (replayed.cache, replayed.table, replayed.taken, replayed.seq)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = replayed.step(x, one, n, 1)
    for t, b in zip((replayed.cache, replayed.table, replayed.taken, replayed.seq), before):
        t.copy_(b)
    for i in range(1, steps + 1):
        x.copy_(qkv[i, :n])
        g.replay()
        assert torch.equal(out, eager.step(qkv[i, :n].clone(), one, n, 1))
    assert torch.equal(replayed.cache, eager.cache) and torch.equal(replayed.table, eager.table)
    assert w4a16.check_device_status() == w4a16.OK


def test_two_streams_with_their_own_workspaces():
    from weight_only_int4_02_gb300 import w4a16
    args = [batch_of(seq, nq, 2, 4, 128, 32, "float16", s) for s, (seq, nq) in enumerate([([9000, 40], [1, 1]), ([3000, 777], [3, 2])])]
    want = [run_and_check(a, 32) for a in args]
    there = [[a[0].cuda()] + [cuda(x) for x in a[1:]] for a in args]
    ws = [torch.zeros(w4a16.kv8_workspace_bytes(), dtype=torch.uint8, device="cuda") for _ in args]
    torch.cuda.synchronize()
    streams, max_q = [torch.cuda.Stream() for _ in args], [1, 3]   # max_q chooses the kernel, and with it the roundings
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(w4a16.kv8_attention(*there[i], 32, max_q[i], return_lse=True, workspace=ws[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_a_list_that_comes_back_to_a_tile_spoils_that_tile_alone():
    from weight_only_int4_02_gb300 import w4a16
    D, heads, page = 128, 2, 16
    k = torch.randn(40, heads, D, device="cuda").to(torch.float16)
    slots = np.concatenate([np.arange(16), np.arange(16, 22), np.arange(20, 24), np.arange(32, 46)])
    cache = w4a16.kv8_cache(4, heads, D, page)
    w4a16.kv8_append(k, k, cuda(slots), cache, page)
    want = ref.append(np.zeros(cache.shape, np.uint8), k.float().cpu().numpy(), k.float().cpu().numpy(), slots, page)
    got = cache.cpu()
    for tile in (0, 2, 3):
        same_cache(got[tile:tile + 1], want[tile:tile + 1], D)


@pytest.mark.parametrize("path", [1, 2])
@pytest.mark.parametrize("heads,group,D", [(1, 128, 128), (16, 8, 64), (3, 1, 128)])
def test_many_heads(path, heads, group, D):
    run_and_check(batch_of([333, 1, 50], [2, 1, 5], heads, group, D, 64, "bfloat16", heads), 64, 0, path)


def test_rows_past_32_bits_of_elements():
    """More than 2^31 elements of queries, and keys behind a stride that passes 32 bits."""
    from weight_only_int4_02_gb300 import w4a16
    T, H, D = 140000, 128, 128
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    q[-100:] = torch.randn(100, H, D, device="cuda").to(torch.bfloat16)
    q[:100] = q[-100:]
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[-100:] = pos[:100] = torch.arange(100, dtype=torch.int32, device="cuda")
    rope = w4a16.rope_table(100, D)
    weight = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    out, _ = w4a16.qk_norm_rope(q, None, pos, rope, q_weight=weight)
    small, _ = w4a16.qk_norm_rope(q[-100:], None, pos[-100:], rope, q_weight=weight)
    assert torch.equal(out[-100:], small) and torch.equal(out[:100], small)
    del out
    wide = q.view(-1, 70000 * H * D)                      # two rows, 2.3 GB apart
    k = wide.as_strided((2, 2, D), (70000 * H * D, D, 1))
    cache, other = (w4a16.kv8_cache(1, 2, D, 16) for _ in range(2))
    k[1].copy_(torch.randn(2, D, device="cuda"))
    for c, x in ((cache, k), (other, k.contiguous())):
        w4a16.kv8_append(x, x, torch.arange(2, device="cuda"), c, 16, positions=pos[:2], rope=rope)
    assert torch.equal(cache, other)


@pytest.mark.parametrize("path", [1, 2])
def test_values_of_a_thousandfold_spread(path):
    """V's scales over a range of 2^10, the largest where the probabilities are small: within the tolerance on either kernel."""
    args = batch_of([700], [40], 1, 2, 128, 16, "float16", 5, spread=0.0)
    q, cache, table, seq, starts = args
    r = np.random.default_rng(1)
    for t in range(0, 700, 16):
        sc = np.array([0.02, 0.02 * 2.0 ** r.integers(-5, 6)], np.float32)
        cache[table[0, t // 16], 0, 0, 32 * 128:32 * 128 + 8] = sc.view(np.uint8)
    run_and_check(args, 16, 0, path)
