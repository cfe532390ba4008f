"""Positions and a key-value cache held in 8 bits: what is measured, and its plain forms.

Three operators of the serving step: queries and keys normed for each head and rotated by their positions in one pass
("norm"), keys rotated and quantised with their values into their slots of an 8-bit paged cache ("append", read back by the
call that reads slots), and attention over that cache ("attention").

Rotation. A table float32 [positions][rot] holds cos(p * base^(-2i / rot)), i < rot / 2, then the sines. Of the first rot
values of a head, pair i is (x[i], x[i + rot / 2]), or (x[2i], x[2i + 1]) where pairs are interleaved:
  (a, b) -> (a cos - b sin, b cos + a sin).
A norm comes before it: x / sqrt(mean(x^2) + eps) * weight.

The cache is one uint8 tensor [pages][kv_heads][page_size / 16][32 * head_dim + 16]. A tile of 16 tokens and head dimension D
holds, in this order:
  K codes   [D/64][16][64]: byte i of token t in slab p is d = 64p + i;
  V codes   [D/64][2][8][4][4][2][2]: byte (p, h, n, c, j, e, i) is d = 64p + 8n + 2j + i of token 8h + 2c + e;
  K scale, V scale  float32, of all 16 tokens;  8 bytes unused.
A stored value is (code - 128) * scale. The tokens of one call that fall into one tile, neighbours there and in the list, are
stored together, K and V alike: with a = max |x| / 127 over their rows (0 below 2^-40, at most 2^40, NaN if a row holds an
infinity or a NaN) and old the tile's scale, 0 if they begin at the tile's first token,
  s = max(old, a), r = 1 / s, code = clamp(rint(x * r), -127, 127) + 128   (s = 0 or NaN: 128),
and where s > old the tile's earlier tokens become clamp(rint((code - 128) * (old * r)), -127, 127) + 128. All of it in 32
bits, each operation rounded by itself.
"""
import math
import random

import torch

own = False

HALF = {"float16": torch.float16, "bfloat16": torch.bfloat16}
DEV = "cuda"
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: the heads of sixteen tokens, slices of a fused projection's output
        dict(name="norm_decode_t16", op="norm", tokens=16, chunks=16, q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, ctx=16384, dtype="float16", lens=31),
        # half of a narrow head rotated, in neighbouring pairs; an odd number of tokens
        dict(name="norm_partial_t1003", op="norm", tokens=1003, chunks=7, q_heads=28, kv_heads=4, dim=64, rot=32,
             interleaved=True, ctx=8192, dtype="bfloat16", lens=32),
        # prompt chunks, many query heads
        dict(name="norm_prompt_t8191", op="norm", tokens=8191, chunks=3, q_heads=64, kv_heads=8, dim=128, rot=128,
             interleaved=False, ctx=32768, dtype="bfloat16", lens=33),
        # one decode step: a token each of sixteen requests into tiles begun before
        dict(name="append_decode_t16", op="append", tokens=16, chunks=16, q_heads=32, kv_heads=32, dim=128, rot=128,
             interleaved=False, ctx=4096, page=16, dtype="float16", lens=41),
        # prompt chunks written to the cache, shared heads
        dict(name="append_prompt_t8191", op="append", tokens=8191, chunks=3, q_heads=64, kv_heads=8, dim=128, rot=128,
             interleaved=False, ctx=16384, page=32, dtype="bfloat16", lens=42),
        # the smallest decode step: one request, latency counts
        dict(name="attention_decode_b1_1k", op="attention", batch=1, q_heads=32, kv_heads=32, dim=128, page=16,
             q_lo=1, q_hi=1, ctx_lo=1000, ctx_hi=1000, window=0, lse=False, dtype="float16", lens=51),
        # a serving batch with ragged lengths, eight query heads to a KV head
        dict(name="attention_decode_b64_ragged", op="attention", batch=64, q_heads=64, kv_heads=8, dim=128, page=32,
             q_lo=1, q_hi=1, ctx_lo=257, ctx_hi=16384, window=0, lse=False, dtype="bfloat16", lens=52),
        # one request with a very long context
        dict(name="attention_decode_b1_128k", op="attention", batch=1, q_heads=32, kv_heads=8, dim=128, page=64,
             q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, window=0, lse=True, dtype="float16", lens=53),
        # drafted tokens checked in one pass, sliding window, narrow heads, unused batch rows
        dict(name="attention_verify_b48_q5", op="attention", batch=48, q_heads=16, kv_heads=4, dim=64, page=16,
             q_lo=1, q_hi=5, ctx_lo=0, ctx_hi=9000, window=4096, lse=True, dtype="bfloat16", lens=54),
        # prompt chunks behind cached context: the matrix products bound it
        dict(name="attention_prompt_b3_q4000", op="attention", batch=3, q_heads=32, kv_heads=8, dim=128, page=32,
             q_lo=777, q_hi=4000, ctx_lo=3001, ctx_hi=8200, window=0, lse=False, dtype="bfloat16", lens=55),
        # a short prompt of narrow heads, full-precision probabilities
        dict(name="attention_prompt_b2_q1000", op="attention", batch=2, q_heads=14, kv_heads=2, dim=64, page=16,
             q_lo=301, q_hi=1000, ctx_lo=301, ctx_hi=2001, window=0, lse=True, dtype="float16", lens=56),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "append", "attention", "attention", "attention", "attention"])
    lens = rng.randrange(1 << 30)
    dtype = rng.choice(["float16", "bfloat16"])
    page = rng.choice([16, 32, 64])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 128])
    if op != "attention":
        tokens = _log(rng, 1, 8191)
        chunks = rng.choice([tokens, _log(rng, 1, tokens), _log(rng, 1, min(tokens, 8))]) if tokens <= 1000 \
            else _log(rng, 1, 64)
        case = dict(op=op, tokens=tokens, chunks=chunks, q_heads=kv * rng.choice([1, 3, 4, 7, 8]), kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 16, 24]), interleaved=rng.choice([False, False, True]),
                    ctx=_log(rng, 16, 32768), dtype=dtype, lens=lens)
        if op == "append":
            case["page"] = page
        return case
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    window = rng.choice([0, 0, _log(rng, 64, 4096)])
    kind = rng.choice(["decode", "verify", "prompt"])
    if kind == "decode":
        b = _log(rng, 1, 100)
        hi = _log(rng, 64, max(64, min(131071, 64 * 8192 // b)))
        q_lo = q_hi = 1
    elif kind == "verify":
        b = _log(rng, 1, 48)
        hi = _log(rng, 64, max(64, min(65536, 48 * 4500 // b)))
        q_lo, q_hi = 1, rng.randint(2, 9)
    else:
        b = rng.randint(1, 3)
        hi = _log(rng, 200, 8200)
        kv, group = rng.choice([1, 2, 4]), rng.choice([1, 4, 7])
        q_lo, q_hi = 1, _log(rng, 17, min(hi, 4000))
    return dict(op=op, batch=b, q_heads=kv * group, kv_heads=kv, dim=dim, page=page, q_lo=q_lo, q_hi=q_hi,
                ctx_lo=rng.choice([0, 1, hi // 4]), ctx_hi=hi, window=window, lse=rng.choice([True, False]),
                dtype=dtype, lens=lens)


def _chunks(case):
    """(new tokens, tokens cached before) of each request of a norm or an append: of the case alone."""
    rng = random.Random(case["lens"])
    t, n = case["tokens"], case["chunks"]
    cuts = sorted(rng.sample(range(1, t), n - 1)) if n > 1 else []
    new = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    return new, [_log(rng, 1, case["ctx"]) - 1 for _ in new]


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each request of an attention: of the case alone."""
    rng = random.Random(case["lens"])
    n = case["batch"]
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
    seq = [_log(rng, max(1, case["ctx_lo"]), case["ctx_hi"]) for _ in range(n)]
    if case["ctx_lo"] == 0 and n > 1:    # an unused row of a static batch: nothing cached, one query
        seq[rng.randrange(n)] = 0
    new[0], seq[0] = case["q_hi"], case["ctx_hi"]
    return [a if s == 0 else min(a, s) for a, s in zip(new, seq)], seq


def _pairs(case):
    """Visible (query, key) pairs and cached tiles that some query sees, over the requests."""
    pairs = tiles = 0
    w = case["window"]
    for a, s in zip(*_lengths(case)):
        if s == 0:
            continue
        first = s - a
        if w == 0:
            pairs += a * (first + 1) + a * (a - 1) // 2
        else:
            pairs += sum(min(w, first + i + 1) for i in range(a))
        low = max(0, first + 1 - w) if w else 0
        tiles += (s - 1) // 16 - low // 16 + 1
    return pairs, tiles


def work(case):
    d = case["dim"]
    if case["op"] == "norm":
        rows = case["tokens"] * (case["q_heads"] + case["kv_heads"])
        return {"bytes": rows * 4 * d + case["tokens"] * (4 * case["rot"] + 4) + 8 * d, "flops": rows * 8 * d}
    if case["op"] == "append":
        rows = case["tokens"] * case["kv_heads"]
        back = sum(b % 16 + a for a, b in zip(*_chunks(case))) * case["kv_heads"]
        # K and V in, table rows, codes out, and the tiles' values read back as 16-bit numbers
        return {"bytes": rows * (4 * d + 2 * d) + case["tokens"] * (4 * case["rot"] + 12) + back * (2 * d + 4 * d),
                "flops": rows * 10 * d}
    pairs, tiles = _pairs(case)
    new, _ = _lengths(case)
    h = case["q_heads"]
    size = tiles * case["kv_heads"] * (32 * d + 8) + 4 * sum(new) * h * d + (4 * sum(new) * h if case["lse"] else 0)
    return {"bytes": size, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------ what a program has in hand
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).to(DEV)


def _starts(lens):
    out = [0]
    for a in lens:
        out.append(out[-1] + a)
    return out


def _codes(shape, g):
    """Codes bell-shaped about 128."""
    normal = torch.erfinv((torch.arange(1024, device=DEV) + 0.5) / 512 - 1) * math.sqrt(2)
    code = (128 + 37 * normal).round().clamp(1, 255).to(torch.uint8)
    return code[torch.randint(0, 1024, shape, generator=g, device=DEV, dtype=torch.int32)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=dict(case), op=case["op"])
    h, kv, d = case["q_heads"], case["kv_heads"], case["dim"]
    dtype = HALF[case["dtype"]]
    width = (h + 2 * kv) * d
    if case["op"] != "attention":
        t, rot = case["tokens"], case["rot"]
        new, before = _chunks(case)
        pos = _ints([b + i for a, b in zip(new, before) for i in range(a)])
        rows = max(a + b for a, b in zip(new, before))
        angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] \
            * BASE ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
        s.update(positions=pos, rope=torch.cat([angle.cos(), angle.sin()], 1).float())
        gain = torch.exp(0.6 * torch.randn(h + 2 * kv, d, generator=g, device=DEV))    # some channels are larger
        x = (torch.randn(t, h + 2 * kv, d, generator=g, device=DEV) * gain).to(dtype).view(t, width)
        s.update(q=x[:, :h * d].view(t, h, d), k=x[:, h * d:(h + kv) * d].view(t, kv, d))
        if case["op"] == "norm":
            s.update(q_weight=(1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dtype),
                     k_weight=(1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dtype))
            return s
        # the chunks' tokens in pages in any order, the tokens before them in the pages' earlier places
        p = case["page"]
        held = [-(-(b % p + a) // p) for a, b in zip(new, before)]
        pages = sum(held) + 3
        ids = torch.randperm(pages, generator=g, device=DEV)

        def slots(first, count):
            """Slots of each request's places first .. first + count of its pages."""
            place = _ints([f + i for f, c in zip(first, count) for i in range(c)], torch.int64)
            page0 = _ints([q for q, c in zip(_starts(held), count) for _ in range(c)], torch.int64)
            return ids[page0 + place // p] * p + place % p

        tile0 = [b % p // 16 * 16 for b in before]
        cache = _codes((pages, kv, p // 16, 32 * d + 16), g)
        old = 0.02 * torch.exp(0.3 * torch.randn(pages, kv, p // 16, 2, generator=g, device=DEV))
        cache[..., 32 * d:32 * d + 8] = old.view(torch.uint8).view(pages, kv, p // 16, 8)
        s.update(v=x[:, (h + kv) * d:].view(t, kv, d), cache=cache, slots=slots([b % p for b in before], new),
                 back=slots(tile0, [b % p - f + a for a, b, f in zip(new, before, tile0)]),
                 runs=sum((b % 16 + a + 15) // 16 for a, b in zip(new, before)))
        return s
    p = case["page"]
    new, seq = _lengths(case)
    cols = max(1, max(-(-b // p) for b in seq))
    held = [-(-b // p) for b in seq]
    pages = sum(held) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    first = _ints(_starts(held), torch.int64)
    col = torch.arange(cols, device=DEV)
    has = col[None] < _ints(held, torch.int64)[:, None]
    table = torch.where(has, ids[(first[:-1, None] + col[None]).clamp(max=pages - 1)], -1).to(torch.int32)
    cache = _codes((pages, kv, p // 16, 32 * d + 16), g)
    scale = 0.02 * torch.exp(0.3 * torch.randn(pages, kv, p // 16, 2, generator=g, device=DEV))
    # tiles past their request's length, and pages that nobody holds, are memory as it was found: NaN
    end = torch.zeros(pages, dtype=torch.int64, device=DEV)
    left = (_ints(seq, torch.int64)[:, None] - col[None] * p).clamp(0, p)
    end[table[has].long()] = left[has]
    stale = (16 * torch.arange(p // 16, device=DEV)[None] >= end[:, None]).view(pages, 1, p // 16, 1)
    scale = torch.where(stale, math.nan, scale)
    cache[..., 32 * d:32 * d + 8] = scale.view(torch.uint8).view(pages, kv, p // 16, 8)
    t = sum(new)
    x = (1.5 * torch.randn(t, width, generator=g, device=DEV)).to(dtype)
    s.update(q=x[:, :h * d].view(t, h, d), cache=cache, table=table, seq=_ints(seq), starts=_ints(_starts(new)),
             max_q=max(new))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        from weight_only_int4_02_gb300 import w4a16
        if s["op"] == "norm":
            return w4a16.qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"], q_weight=s["q_weight"],
                                      k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        if s["op"] == "append":
            w4a16.kv8_append(s["k"], s["v"], s["slots"], s["cache"], c["page"], positions=s["positions"], rope=s["rope"],
                             interleaved=c["interleaved"])
            return w4a16.kv8_read(s["cache"], s["back"], c["page"], dtype=s["k"].dtype)
        return w4a16.kv8_attention(s["q"], s["cache"], s["table"], s["seq"], s["starts"], c["page"], s["max_q"],
                                   window=c["window"], return_lse=c["lse"])
    return {"norm": _norm, "append": _append, "attention": _attention}[s["op"]](s, c)


# ------------------------------------------------------------------ plain forms
def _rotated(x, positions, rope, interleaved):
    """x float32 [tokens][heads][d], rotated; each product and sum rounded by itself."""
    rot = rope.shape[1]
    at = rope[positions.long()][:, None]
    cos, sin = at[..., :rot // 2], at[..., rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    y = [a * cos - b * sin, b * cos + a * sin]
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _norm(s, c):
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_rotated(y, s["positions"], s["rope"], c["interleaved"]).to(x.dtype))
    return out


def _places(tok, d):
    """Bytes of a tile that hold a token's codes, [tokens][d] each: K's and V's."""
    i = torch.arange(d, device=DEV)
    p, r = i // 64, i % 64
    k = (p * 16 + tok[:, None]) * 64 + r
    h, c, e = tok[:, None] // 8, tok[:, None] % 8 // 2, tok[:, None] % 2
    v = 16 * d + ((((p * 2 + h) * 8 + r // 8) * 4 + c) * 4 + r % 8 // 2) * 4 + 2 * e + r % 2
    return k, v


def _append(s, c):
    p, d, cache, slots = c["page"], c["dim"], s["cache"], s["slots"]
    kv, size = cache.shape[1], cache.shape[3]
    flat = cache.view(-1)
    four = torch.arange(4, device=DEV)
    heads = torch.arange(kv, device=DEV)

    def base(tile):                                                # bytes of a tile of each head, [..][kv]
        page, in_page = tile // (p // 16), tile % (p // 16)
        return ((page[:, None] * kv + heads) * (p // 16) + in_page[:, None]) * size

    # runs of tokens that are neighbours in a tile
    ahead = torch.cat([slots.new_full((1,), -2), slots[:-1]])
    begins = (slots != ahead + 1) | (slots % 16 == 0)
    run = torch.cumsum(begins, 0) - 1
    first = torch.sort(begins.to(torch.uint8), descending=True, stable=True).indices[:s["runs"]]
    tile, offset = slots[first] // 16, slots[first] % 16
    k_old, v_old = _places(torch.arange(16, device=DEV), d)        # [16][d]
    k_new, v_new = _places(slots % 16, d)                          # [tokens][d]
    k = _rotated(s["k"].float(), s["positions"], s["rope"], c["interleaved"])
    for x, old_at, new_at, scale_at in ((k, k_old, k_new, 32 * d), (s["v"].float(), v_old, v_new, 32 * d + 4)):
        top = x.abs().amax(-1)                                     # [tokens][kv]
        most = torch.zeros(s["runs"], kv, device=DEV).scatter_reduce(0, run[:, None].expand(-1, kv), top, "amax")
        a = most / 127.0
        a = torch.where(a < 2.0 ** -40, 0.0, a).clamp(max=2.0 ** 40)
        a = torch.where(most <= 3.4028234663852886e38, a, math.nan)
        at = base(tile)[..., None] + scale_at + four
        old = flat[at].contiguous().view(torch.float32).view(-1, kv)
        old = torch.where(offset[:, None] == 0, 0.0, old)
        scale = torch.maximum(old, a)
        r = torch.where(scale > 0, 1.0 / scale, 0.0)
        bytes_ = base(tile)[..., None, None] + old_at              # [runs][kv][16][d]
        code = flat[bytes_]
        less = torch.round((code.float() - 128) * (old * r)[..., None, None]).clamp(-127, 127) + 128
        before = torch.arange(16, device=DEV)[:, None] < offset[:, None, None, None]
        again = before & (scale > old)[..., None, None]
        flat[bytes_] = torch.where(again, less.to(torch.uint8), code)
        code = torch.round(x * r[run][..., None]).clamp(-127, 127) + 128
        code = torch.where(scale[run][..., None] > 0, code, 128.0)
        flat[base(slots // 16)[..., None] + new_at[:, None]] = code.to(torch.uint8)
        flat[at] = scale[..., None].view(torch.uint8).view(-1, kv, 4)
    back = s["back"]
    out = []
    for which, scale_at in ((0, 32 * d), (1, 32 * d + 4)):
        code = flat[base(back // 16)[..., None] + _places(back % 16, d)[which][:, None]].float() - 128
        scale = flat[base(back // 16)[..., None] + scale_at + four].contiguous().view(torch.float32)
        out.append((code * scale).to(s["k"].dtype))
    return out


def _attention(s, c):
    p, d, kv, h = c["page"], c["dim"], c["kv_heads"], c["q_heads"]
    table, seq, starts, q = s["table"].long(), s["seq"].long(), s["starts"].long(), s["q"]
    n, cols, t, m, group = table.shape[0], table.shape[1], q.shape[0], s["max_q"], h // kv
    length = cols * p
    tiles = length // 16
    raw = s["cache"][table.clamp(min=0)].transpose(1, 2).reshape(n, kv, tiles, 32 * d + 16)
    scale = raw[..., 32 * d:32 * d + 8].contiguous().view(torch.float32)         # [n][kv][tiles][2]
    seen = torch.arange(length, device=DEV)[None] < seq[:, None]                # [n][length]
    ok = seen[:, None, :, None]

    def value(code, which):
        x = (code.reshape(n, kv, tiles, 16 * d).float() - 128) * scale[..., which, None]
        return torch.where(ok, x.reshape(n, kv, length, d), 0.0)

    k = value(raw[..., :16 * d].view(n, kv, tiles, d // 64, 16, 64).transpose(3, 4), 0)
    code = raw[..., 16 * d:32 * d].view(n, kv, tiles, d // 64, 2, 8, 4, 4, 2, 2)
    v = value(code.permute(0, 1, 2, 4, 6, 8, 3, 5, 7, 9), 1)
    del raw, code
    i = torch.arange(m, device=DEV)
    at = (starts[:-1, None] + i).clamp(max=max(t - 1, 0))                       # [n][m]
    qs = q[at].float().view(n, m, kv, group, d).permute(0, 2, 3, 1, 4).reshape(n, kv, group * m, d)
    score = ((qs @ k.transpose(-1, -2)) * (1.0 / math.sqrt(d))).view(n, kv, group, m, length)
    count = starts[1:] - starts[:-1]
    pos = (seq - count)[:, None] + i                                            # [n][m]
    key = torch.arange(length, device=DEV)
    mask = (key <= pos[..., None]) & seen[:, None]
    if c["window"]:
        mask &= key > pos[..., None] - c["window"]
    score = torch.where(mask[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    del score
    total = e.sum(-1, keepdim=True)
    o = (e.view(n, kv, group * m, length) @ v).view(n, kv, group, m, d) / torch.where(total == 0, 1.0, total)
    row = torch.searchsorted(starts[1:].contiguous(), torch.arange(t, device=DEV), right=True)
    j = torch.arange(t, device=DEV) - starts[row]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, m, h, d)[row, j].to(q.dtype)
    if not c["lse"]:
        return o
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(n, m, h)
    return [o, lse[row, j]]


# ------------------------------------------------------------------ the definition, in 64 bits
def _turned(x, s, interleaved):
    """x float64, rotated as complex numbers."""
    rot = s["rope"].shape[1]
    at = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(at[:, :rot // 2], at[:, rot // 2:])[:, None]
    y = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out = []
        for x, w in (("q", "q_weight"), ("k", "k_weight")):
            y = s[x].double()
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / case["dim"] + EPS) * s[w].double()
            out.append(_turned(y, s, case["interleaved"]))
        return out
    d, kv, p = case["dim"], case["kv_heads"], case["page"]
    if case["op"] == "append":
        if case["chunks"] > 200:
            return None
        new, before = _chunks(case)
        out = []
        for which, x in enumerate((_turned(s["k"].double(), s, case["interleaved"]), s["v"].double())):
            rows, at, back_at = [], 0, 0
            for a, b in zip(new, before):
                held, o = b % 16, 0
                while o < a:                                       # tile by tile
                    take = min(16 - held, a - o)
                    y = x[at + o:at + o + take]                    # [take][kv][d]
                    scale = (y.abs().amax(-1).amax(0) / 127).float().double()          # [kv]
                    if held:
                        slot = int(s["back"][back_at])
                        raw = s["cache"][slot // p, :, slot % p // 16]                 # [kv][bytes]
                        old = raw[:, 32 * d + 4 * which:32 * d + 4 * which + 4].contiguous().view(torch.float32).double()[:, 0]
                        c = raw[:, 16 * d * which:16 * d * (which + 1)].double() - 128
                        c = c.view(kv, d // 64, 16, 64).transpose(1, 2).reshape(kv, 16, d) if which == 0 else \
                            c.view(kv, d // 64, 2, 8, 4, 4, 2, 2).permute(0, 2, 4, 6, 1, 3, 5, 7).reshape(kv, 16, d)
                        scale = torch.maximum(scale, old)
                        c = torch.round(c * (old / scale)[:, None, None])
                        rows.append((c * scale[:, None, None]).transpose(0, 1)[:held])
                    rows.append(torch.round(y / scale[:, None]).clamp(-127, 127) * scale[:, None])
                    o, back_at, held = o + take, back_at + held + take, 0
                at += a
            out.append(torch.cat(rows))
        return out
    new, seq = _lengths(case)
    h, t = case["q_heads"], sum(new)
    o = torch.zeros(t, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (a, n) in enumerate(zip(new, seq)):
        first, at = at, at + a
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // p)].long()
        for g in range(kv):
            raw = s["cache"][pages, g].reshape(-1, 32 * d + 16)                 # [tiles][bytes]
            scale = raw[:, 32 * d:32 * d + 8].contiguous().view(torch.float32).double()
            kc, vc = raw[:, :16 * d].view(-1, d // 64, 16, 64), raw[:, 16 * d:32 * d].view(-1, d // 64, 2, 8, 4, 4, 2, 2)
            key = torch.cat([kc[:, j] for j in range(d // 64)], -1).double() - 128          # [tiles][16][d]
            val = torch.stack([vc[:, :, tok // 8, :, tok % 8 // 2, :, tok % 2].reshape(-1, d) for tok in range(16)], 1).double() - 128
            key = (key * scale[:, 0, None, None]).view(-1, d)[:n]
            val = (val * scale[:, 1, None, None]).view(-1, d)[:n]
            pos = torch.arange(n - a, n, device=DEV)[:, None]
            col = torch.arange(n, device=DEV)[None]
            see = (col <= pos) if not case["window"] else (col <= pos) & (col > pos - case["window"])
            for head in range(g * (h // kv), (g + 1) * (h // kv)):
                x = s["q"][first:at, head].double() @ key.T / math.sqrt(d)
                x = x.masked_fill(~see, -math.inf)
                lse[first:at, head] = torch.logsumexp(x, -1)
                o[first:at, head] = torch.softmax(x, -1) @ val
    return [o, lse] if case["lse"] else o
