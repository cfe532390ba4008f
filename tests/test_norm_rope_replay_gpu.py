"""Norms and rotations captured into a graph: what a replay reads is what is there when it runs."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("what", ["positions", "rope", "weight", "x"])
def test_a_replay_takes_what_has_changed(what, interleaved):
    from weight_only_int4_02_gb300 import w4a16
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, H, KV, D = 37, 12, 4, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(T, H + KV, D, generator=g, device="cuda").to(torch.bfloat16)
    there = dict(positions=torch.arange(T, dtype=torch.int32, device="cuda") * 7, rope=w4a16.rope_table(300, D),
                 weight=(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16), x=x)

    def call(**outs):
        return w4a16.qk_norm_rope(x[:, :H], x[:, H:], there["positions"], there["rope"], q_weight=there["weight"], k_weight=there["weight"],
                                  interleaved=interleaved, **outs)

    old = [t.clone() for t in call()]
    out = [torch.zeros_like(t) for t in old]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q_out=out[0], k_out=out[1])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, old))
    if what == "positions":
        there[what].add_(3)
    else:
        there[what].mul_(-0.5)
    graph.replay()
    for a, b, before in zip(out, call(), old):
        assert torch.equal(a, b) and not torch.equal(a, before)
