"""A small decoder served with this library: 4-bit weights, a key-value cache in 4 or 8 bits, sampling.

Shows the serving step's calls together, as a server would make them: block tables and slot maps
from the batch's lengths (kv4_tables), the projections (gemm), queries and keys normed for each head and
rotated by their positions (qk_norm_rope), new keys and values into their slots (kv4_append, or kv8_append, which
rotates keys on the way), attention over the cache (kv4_attention, kv8_attention), the MLP (gemm_fused) and the next
tokens (sample). Weights are random; requests join with prompts of their own lengths and decode
together. The hidden state's norms and the embedding are plain torch.

    python -m weight_only_int4_02_gb300.serve --requests 4 --steps 16
    python -m weight_only_int4_02_gb300.serve --cache-bits 8 --rope-base 10000 --qk-norm
"""
import argparse
import time

import torch

from . import w4a16

GROUP = 128


class Linear:
    """A [K][N] weight in 4 bits: codes uniform on 0..15, scales that keep outputs near the inputs' size."""

    def __init__(self, K, N, generator, device):
        codes = torch.randint(0, 16, (K, N), generator=generator, device=device, dtype=torch.uint8)
        std = 4.6 * K ** 0.5      # of a sum of K codes about the zero-point, for inputs of size one
        scales = (0.5 + torch.rand(K // GROUP, N, generator=generator, device=device)) / std
        self.N = N
        self.packed, self.scales = w4a16.pack(codes, scales.to(torch.float16), GROUP)

    def __call__(self, x, residual=None, activation="none"):
        return w4a16.gemm_fused(x, self.packed, self.scales, self.N, GROUP, residual=residual, activation=activation)


def rms_norm(x):
    x32 = x.float()
    return (x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Decoder:
    """hidden = q_heads * head_dim; query heads share KV heads in groups. cache_bits: 4 or 8; rope_base: queries and keys
    are rotated by their positions, up to max_positions (None: they are not); qk_norm: and normed for each head."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, head_dim=128, ffn=2048, vocab=4096, seed=0, device="cuda", cache_bits=4,
                 rope_base=None, max_positions=4096, qk_norm=False):
        if cache_bits not in (4, 8):
            raise ValueError("a cache of 4 or 8 bits, not %r" % (cache_bits,))
        g = torch.Generator(device=device).manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.vocab = q_heads, kv_heads, head_dim, vocab
        hidden = q_heads * head_dim
        self.embedding = torch.randn(vocab, hidden, generator=g, device=device).to(torch.float16)
        self.layers = [dict(qkv=Linear(hidden, hidden + 2 * kv_heads * head_dim, g, device), out=Linear(hidden, hidden, g, device),
                            up=Linear(hidden, ffn, g, device), down=Linear(ffn, hidden, g, device)) for _ in range(layers)]
        self.head = Linear(hidden, vocab, g, device)
        self.cache_bits, self.max_positions = cache_bits, max_positions
        self.rope = None if rope_base is None else w4a16.rope_table(max_positions, head_dim, rope_base, device=device)
        if qk_norm:
            for layer in self.layers:
                layer["q_norm"], layer["k_norm"] = ((1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).to(torch.float16)
                                                    for _ in range(2))

    def caches(self, pages, page_size):
        make = w4a16.kv4_cache if self.cache_bits == 4 else w4a16.kv8_cache
        return [make(pages, self.kv_heads, self.head_dim, page_size) for _ in self.layers]

    def attention(self, layer, qkv, cache, table, seq_lens, slots, starts, page_size, max_q, positions):
        """Attention's output of new tokens, their keys and values stored: qkv [tokens][q_heads + 2 kv_heads][head_dim]."""
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)   # slices of it need no copy
        norms = dict(q_weight=layer.get("q_norm"), k_weight=layer.get("k_norm"))
        late = self.cache_bits == 8 and norms["k_weight"] is None   # keys without a norm are rotated as they are stored
        if self.rope is not None or norms["q_weight"] is not None:
            if late:
                w4a16.qk_norm_rope(q, None, positions, self.rope, q_out=q)
            else:
                w4a16.qk_norm_rope(q, k, positions if self.rope is not None else None, self.rope, q_out=q, k_out=k, **norms)
        if self.cache_bits == 4:
            w4a16.kv4_append(k, v, slots, cache, page_size)
            return w4a16.kv4_attention(q, cache, table, seq_lens, starts, page_size, max_q)
        turn = dict(positions=positions, rope=self.rope) if late and self.rope is not None else {}
        w4a16.kv8_append(k, v, slots, cache, page_size, **turn)
        return w4a16.kv8_attention(q, cache, table, seq_lens, starts, page_size, max_q)

    def step(self, tokens, caches, table, seq_lens, slots, starts, page_size, max_q, positions=None):
        """Logits of the last token of each request: tokens int64 [new tokens of the batch]; positions, as kv4_tables gives them,
        are wanted where the model rotates."""
        if self.rope is not None and positions is None:
            raise ValueError("a model that rotates wants its tokens' positions")
        q_heads, kv, d = self.q_heads, self.kv_heads, self.head_dim
        x = self.embedding[tokens]
        for layer, cache in zip(self.layers, caches):
            qkv = layer["qkv"](rms_norm(x)).view(-1, q_heads + 2 * kv, d)
            a = self.attention(layer, qkv, cache, table, seq_lens, slots, starts, page_size, max_q, positions)
            x = layer["out"](a.view(-1, q_heads * d), residual=x)
            x = layer["down"](layer["up"](rms_norm(x), activation="silu"), residual=x)
        return self.head(rms_norm(x[starts[1:].long() - 1]))


def generate(model, prompts, steps, page_size=16, max_len=512, temperature=0.8, top_k=50, top_p=0.95, seed=0):
    """Tokens drawn for each prompt (a list of int64 CUDA tensors): int32 [requests][steps]. max_len: cached
    tokens that a request may come to hold (its prompt and every drawn token but the last), up to whole pages."""
    cols = -(-max_len // page_size)
    if not prompts or min(len(p) for p in prompts) == 0:
        raise ValueError("generate wants a prompt of at least one token for every request")
    if max(len(p) for p in prompts) + steps - 1 > cols * page_size:
        raise ValueError("a prompt of %d tokens and %d steps do not fit the %d tokens of max_len's pages" %
                         (max(len(p) for p in prompts), steps, cols * page_size))
    if model.rope is not None and max(len(p) for p in prompts) + steps - 1 > model.max_positions:
        raise ValueError("a prompt of %d tokens and %d steps pass the model's %d positions" %
                         (max(len(p) for p in prompts), steps, model.max_positions))
    n, device = len(prompts), prompts[0].device
    caches = model.caches(n * cols, page_size)
    table = torch.full((n, cols), -1, dtype=torch.int32, device=device)
    free = torch.randperm(n * cols, device=device).to(torch.int32)
    taken = torch.zeros(1, dtype=torch.int32, device=device)
    g = torch.Generator(device=device).manual_seed(seed)
    uniform = torch.rand(steps, n, generator=g, device=device)
    settings = (torch.full((n,), temperature, device=device), torch.full((n,), top_k, dtype=torch.int32, device=device),
                torch.full((n,), top_p, device=device))
    new = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=device)
    one = torch.ones_like(new)
    seq_lens, tokens, max_q = torch.zeros_like(new), torch.cat(prompts), max(len(p) for p in prompts)
    drawn = []
    for step in range(steps):
        seq_lens = seq_lens + new
        slots, positions, starts, taken = w4a16.kv4_tables(seq_lens, new, free, table, page_size, tokens.numel(), taken=taken)
        logits = model.step(tokens, caches, table, seq_lens, slots, starts, page_size, max_q, positions)
        token, _ = w4a16.sample(logits, uniform[step], *settings)
        drawn.append(token)
        tokens, new, max_q = token.long(), one, 1
    return torch.stack(drawn, 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=100, help="tokens of the longest prompt")
    ap.add_argument("--cache-bits", type=int, default=4, choices=(4, 8), help="bits of the key-value cache")
    ap.add_argument("--rope-base", type=float, default=None, help="rotate queries and keys by their positions, with this base")
    ap.add_argument("--qk-norm", action="store_true", help="norm queries and keys for each head")
    a = ap.parse_args()
    model = Decoder(layers=a.layers, cache_bits=a.cache_bits, rope_base=a.rope_base, qk_norm=a.qk_norm,
                    max_positions=a.prompt + a.steps)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randint(0, model.vocab, (max(1, a.prompt - 13 * i),), generator=g, device="cuda") for i in range(a.requests)]
    max_len = a.prompt + a.steps
    generate(model, prompts, min(a.steps, 2), max_len=max_len)
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens = generate(model, prompts, a.steps, max_len=max_len)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(tokens.tolist())
    print("%d tokens for each of %d requests in %.1f ms" % (a.steps, a.requests, t * 1e3))
    if w4a16.check_device_status() != w4a16.OK:
        raise SystemExit("a kernel's wait timed out")


if __name__ == "__main__":
    main()
