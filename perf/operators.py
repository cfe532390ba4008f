"""The serving step over a key-value cache held in 4 bits: what is measured, and its plain forms.

Four operators, in the order in which a step runs them: the block tables and slot maps of a
batch built from its request lengths ("tables"), new keys and values quantised into their
slots ("append"), attention over the 4-bit cache ("attention"), and sampling of the next
token from the logits ("sample").

The cache is one uint8 tensor [pages][kv_heads][page_size / 16][16 * (head_dim + 6)]. A tile
of 16 tokens and head dimension D holds, in this order:
  K codes   [16][D/2]: byte j of a token holds d = 2j in bits 0..3 and d = 2j + 1 in bits 4..7;
  V codes   [2][8][4][D/32][2] 16-bit words: word (h, n, c, w, e) holds, in nibble i (bits
            4i..4i+3), d = n*D/8 + 4w + i of token 8h + 2c + e;
  K scales  binary16 [16];  V scales  binary16 [16];  K zero-points  uint8 [16];  V zero-points.
A stored value is (code - zero) * scale. A row x of D values is stored with
  lo = min(x, 0), hi = max(x, 0), s = fp16(min((hi - lo) / 15, 65504)), r = 1 / s,
  z = clamp(rint(-lo * r), 0, 15), code = clamp(rint(x * r) + z, 0, 15)   (s = 0: all zero),
and with scale NaN if it holds an infinity or a NaN.
"""
import math
import random

import torch

own = False

HALF = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: eight requests, one new token each
        dict(name="tables_decode_b8", op="tables", batch=8, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=2048, page=16,
             max_pages=256, lens=11),
        # a continuous batch: a thousand requests, most decoding, some with a prompt chunk
        dict(name="tables_mixed_b1000", op="tables", batch=1000, new_lo=0, new_hi=512, ctx_lo=1, ctx_hi=32768, page=32,
             max_pages=1024, lens=12),
        # the keys and values of a decode step, slices of a fused projection's output
        dict(name="append_decode_t16", op="append", tokens=16, q_heads=32, kv_heads=32, dim=128, page=16,
             dtype="float16"),
        # a prompt chunk written to the cache, shared heads
        dict(name="append_prompt_t8191", op="append", tokens=8191, q_heads=64, kv_heads=8, dim=128, page=32,
             dtype="bfloat16"),
        # the smallest decode step: one request, latency counts
        dict(name="attention_decode_b1_1k", op="attention", batch=1, q_heads=32, kv_heads=32, dim=128, page=16,
             q_lo=1, q_hi=1, ctx_lo=1000, ctx_hi=1000, window=0, lse=False, dtype="float16", lens=21),
        # a serving batch with ragged lengths, eight query heads to a KV head
        dict(name="attention_decode_b64_ragged", op="attention", batch=64, q_heads=64, kv_heads=8, dim=128, page=32,
             q_lo=1, q_hi=1, ctx_lo=257, ctx_hi=16384, window=0, lse=False, dtype="bfloat16", lens=22),
        # one request with a very long context
        dict(name="attention_decode_b1_128k", op="attention", batch=1, q_heads=32, kv_heads=8, dim=128, page=64,
             q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, window=0, lse=True, dtype="float16", lens=23),
        # drafted tokens checked in one pass, sliding window, narrow heads, unused batch rows
        dict(name="attention_verify_b48_q5", op="attention", batch=48, q_heads=16, kv_heads=4, dim=64, page=16,
             q_lo=1, q_hi=5, ctx_lo=0, ctx_hi=9000, window=4096, lse=True, dtype="bfloat16", lens=24),
        # prompt chunks behind cached context: the matrix products bound it
        dict(name="attention_prompt_b3_q4000", op="attention", batch=3, q_heads=32, kv_heads=8, dim=128, page=32,
             q_lo=777, q_hi=4000, ctx_lo=3001, ctx_hi=8200, window=0, lse=False, dtype="bfloat16", lens=25),
        # one row of logits
        dict(name="sample_b1_v32000", op="sample", batch=1, vocab=32000, dtype="float16", mix="usual"),
        # a serving batch, each row with its own settings
        dict(name="sample_b128_v131072", op="sample", batch=128, vocab=131072, dtype="bfloat16", mix="mixed"),
        # full-precision logits of an odd vocabulary, with masked tokens
        dict(name="sample_b256_v100003", op="sample", batch=256, vocab=100003, dtype="float32", mix="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "attention", "sample"])
    lens = rng.randrange(1 << 30)
    dtype = rng.choice(["float16", "bfloat16"])
    page = rng.choice([16, 32, 64])
    if op == "tables":
        hi = _log(rng, 512, 32768)
        return dict(op=op, batch=_log(rng, 1, 1000), new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, 512),
                    ctx_lo=1, ctx_hi=hi, page=page, max_pages=-(-(hi + 512) // page), lens=lens)
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 128])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8191), q_heads=kv * rng.choice([1, 4, 8]), kv_heads=kv, dim=dim,
                    page=page, dtype=dtype)
    if op == "sample":
        return dict(op=op, batch=_log(rng, 1, 200), vocab=_log(rng, 1000, 100003),
                    dtype=rng.choice(["float16", "bfloat16", "float32"]), mix=rng.choice(["usual", "mixed"]))
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


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each request: of the case alone, so that work() knows them."""
    rng = random.Random(case["lens"])
    n = case["batch"]
    if case["op"] == "tables":
        new = [rng.choice([case["new_lo"], 1, 1, 1, rng.randint(case["new_lo"], case["new_hi"])])
               if case["new_hi"] > 1 else 1 for _ in range(n)]
        seq = [a + _log(rng, case["ctx_lo"], case["ctx_hi"] + 1) - 1 for a in new]
    else:
        new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(n)]
        seq = [_log(rng, max(1, case["ctx_lo"]), case["ctx_hi"]) for _ in range(n)]
        if case["ctx_lo"] == 0 and n > 1:    # an unused row of a static batch: nothing cached, one query
            seq[rng.randrange(n)] = 0
        new[0], seq[0] = case["q_hi"], case["ctx_hi"]
        new = [a if s == 0 else min(a, s) for a, s in zip(new, seq)]
    return new, seq


def _pairs(case):
    """Visible (query, key) pairs and cached tokens that some query sees, over the requests."""
    pairs = tokens = 0
    w = case["window"]
    for a, s in zip(*_lengths(case)):
        if s == 0:
            continue
        first = s - a
        if w == 0:
            pairs += a * (first + 1) + a * (a - 1) // 2
            tokens += s
        else:
            pairs += sum(min(w, first + i + 1) for i in range(a))
            tokens += s - max(0, first + 1 - w)
    return pairs, tokens


def work(case):
    if case["op"] == "tables":
        new, _ = _lengths(case)
        n = case["batch"]
        return {"bytes": 12 * n + 4 + 4 * n * case["max_pages"] + 12 * sum(new), "flops": 0}
    if case["op"] == "append":
        rows = case["tokens"] * case["kv_heads"]
        d = case["dim"]
        # K and V in, blocks out, and the stored values read back as 16-bit numbers
        return {"bytes": rows * (4 * d + 2 * (d + 6) + 4 * d) + 16 * case["tokens"], "flops": rows * 10 * d}
    if case["op"] == "attention":
        pairs, tokens = _pairs(case)
        new, _ = _lengths(case)
        d, h = case["dim"], case["q_heads"]
        size = tokens * case["kv_heads"] * (d + 6) + 4 * sum(new) * h * d + (4 * sum(new) * h if case["lse"] else 0)
        return {"bytes": size, "flops": 4 * pairs * h * d}
    size = 4 if case["dtype"] == "float32" else 2
    n = case["batch"] * case["vocab"]
    return {"bytes": n * size + 28 * case["batch"], "flops": 4 * n}


# ------------------------------------------------------------------ what a program has in hand
def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).to(DEV)


def _starts(lens):
    out = [0]
    for a in lens:
        out.append(out[-1] + a)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=dict(case), op=case["op"])
    if case["op"] == "tables":
        new, seq = _lengths(case)
        p, cols = case["page"], case["max_pages"]
        old = _ints([min(cols, -(-(b - a) // p)) for a, b in zip(new, seq)], torch.int64)
        need = sum(min(cols, -(-b // p)) for b in seq)
        ids = torch.randperm(need + 37, generator=g, device=DEV).to(torch.int32)
        held = int(old.sum())
        col = torch.arange(cols, device=DEV)
        has = col[None] < old[:, None]
        at = (torch.cumsum(old, 0) - old)[:, None] + col[None]
        table = torch.where(has, ids[at.clamp(max=need)], -1).to(torch.int32)
        s.update(new=_ints(new), seq=_ints(seq), table=table, free=ids[held:].contiguous(), tokens=sum(new),
                 taken=torch.zeros(1, dtype=torch.int32, device=DEV))
        return s
    if case["op"] == "sample":
        n, v = case["batch"], case["vocab"]
        x = torch.randn(n, v, generator=g, device=DEV) * 2.0
        near = torch.randint(0, v, (n, 24), generator=g, device=DEV)
        x.scatter_(1, near, 8.0 + 3.0 * torch.randn(n, 24, generator=g, device=DEV))
        temp = torch.full((n,), 0.8, device=DEV)
        top_k = torch.full((n,), 50, dtype=torch.int32, device=DEV)
        top_p = torch.full((n,), 0.95, device=DEV)
        min_p = torch.zeros(n, device=DEV)
        if case["mix"] == "mixed":
            kind = torch.arange(n, device=DEV) % 6
            temp = torch.where(kind == 1, 0.0, 0.5 + torch.rand(n, generator=g, device=DEV))      # greedy rows
            top_k = torch.where(kind == 2, 0, torch.randint(1, 1000, (n,), generator=g, device=DEV)).to(torch.int32)
            top_p = torch.where((kind == 2) | (kind == 3), 1.0, 0.5 + 0.5 * torch.rand(n, generator=g, device=DEV))
            top_k = torch.where(kind == 4, 0, top_k).to(torch.int32)                                # top-p alone
            min_p = torch.where(kind == 5, 0.05, 0.0)
            masked = torch.rand(n, v, generator=g, device=DEV) < 0.5                               # a grammar's mask
            x = torch.where(masked & (kind == 3)[:, None], -math.inf, x)
        u = torch.rand(n, generator=g, device=DEV)
        s.update(logits=x.to(HALF[case["dtype"]]), temp=temp, top_k=top_k, top_p=top_p, min_p=min_p, u=u)
        return s
    h, kv, d, p = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    tile = 16 * (d + 6)
    dtype = HALF[case["dtype"]]
    width = (h + 2 * kv) * d
    if case["op"] == "append":
        t = case["tokens"]
        pages = -(-t // p) + 8
        gain = torch.exp(0.6 * torch.randn(2 * kv, d, generator=g, device=DEV))    # some channels are larger
        x = torch.randn(t, h + 2 * kv, d, generator=g, device=DEV)
        x[:, h:] *= gain
        x = x.to(dtype).view(t, width)
        slots = torch.randperm(pages * p, generator=g, device=DEV)[:t].to(torch.int64)
        s.update(k=x[:, h * d:(h + kv) * d].view(t, kv, d), v=x[:, (h + kv) * d:].view(t, kv, d), slots=slots,
                 cache=torch.zeros(pages, kv, p // 16, tile, dtype=torch.uint8, device=DEV))
        return s
    new, seq = _lengths(case)
    cols = max(1, max(-(-b // p) for b in seq))
    held = [-(-b // p) for b in seq]
    pages = sum(held) + 3
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    first = _ints(_starts(held), torch.int64)
    col = torch.arange(cols, device=DEV)
    has = col[None] < _ints(held, torch.int64)[:, None]
    table = torch.where(has, ids[(first[:-1, None] + col[None]).clamp(max=pages - 1)], -1).to(torch.int32)
    # codes bell-shaped about the zero-point, scales log-normal about 0.25
    normal = torch.erfinv((torch.arange(256, device=DEV) + 0.5) / 128 - 1) * math.sqrt(2)
    nib = (7.5 + 2.6 * normal).round().clamp(0, 15).to(torch.uint8)
    cache = torch.empty(pages, kv, p // 16, tile, dtype=torch.uint8, device=DEV)
    shape = (pages, kv, p // 16, 16 * d)
    cache[..., :16 * d] = nib[torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.int32)]
    cache[..., :16 * d] |= nib[torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.int32)] << 4
    scale = torch.exp(0.3 * torch.randn(pages, kv, p // 16, 2, 16, generator=g, device=DEV)) * 0.25
    # a page's tokens past its request's length, and pages that nobody holds, are memory as it was found: NaN
    end = torch.full((pages,), 0, dtype=torch.int64, device=DEV)
    left = (_ints(seq, torch.int64)[:, None] - col[None] * p).clamp(0, p)
    end[table[has].long()] = left[has]
    stale = (torch.arange(p, device=DEV)[None] >= end[:, None]).view(pages, 1, p // 16, 1, 16)
    scale = torch.where(stale, math.nan, scale).to(torch.float16)
    cache[..., 16 * d:16 * d + 64] = scale.view(torch.uint8).view(pages, kv, p // 16, 64)
    cache[..., 16 * d + 64:] = torch.randint(5, 11, (pages, kv, p // 16, 32), generator=g, device=DEV, dtype=torch.uint8)
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
        if s["op"] == "tables":
            slots, positions, starts, taken = w4a16.kv4_tables(s["seq"], s["new"], s["free"], s["table"], c["page"],
                                                               s["tokens"], taken=s["taken"])
            return [s["table"], slots, positions, starts, taken]
        if s["op"] == "append":
            w4a16.kv4_append(s["k"], s["v"], s["slots"], s["cache"], c["page"])
            return w4a16.kv4_read(s["cache"], s["slots"], c["page"], dtype=s["k"].dtype)
        if s["op"] == "attention":
            return w4a16.kv4_attention(s["q"], s["cache"], s["table"], s["seq"], s["starts"], c["page"], s["max_q"],
                                       window=c["window"], return_lse=c["lse"])
        return w4a16.sample(s["logits"], s["u"], s["temp"], s["top_k"], s["top_p"], s["min_p"])
    return {"tables": _tables, "append": _append, "attention": _attention, "sample": _sample}[s["op"]](s, c)


# ------------------------------------------------------------------ plain forms
def _tables(s, c):
    seq, new, free = s["seq"].long(), s["new"].long().clamp(min=0), s["free"]
    p, cols, t = c["page"], s["table"].shape[1], s["tokens"]
    old = (((seq - new).clamp(min=0) + p - 1) // p).clamp(max=cols)
    want = ((seq + p - 1) // p).clamp(max=cols)
    fresh = (want - old).clamp(min=0)
    end = torch.cumsum(fresh, 0) + s["taken"].long()
    col = torch.arange(cols, device=DEV)[None]
    at = (end - fresh)[:, None] + col - old[:, None]
    taken_page = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where(col < old[:, None], s["table"], torch.where(col < want[:, None], taken_page, -1))
    table = table.to(torch.int32)
    last = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), last])
    i = torch.arange(t, device=DEV)
    row = torch.searchsorted(last, i, right=True).clamp(max=seq.numel() - 1)
    pos = seq[row] - new[row] + i - starts[row]
    page = table[row, (pos // p).clamp(0, cols - 1)].long()
    fine = (pos >= 0) & (pos // p < cols) & (page >= 0)
    slots = torch.where(fine, page * p + pos % p, -1)
    return [table, slots, pos.to(torch.int32), starts.to(torch.int32), end[-1:].to(torch.int32)]


def _quantise(x):
    """Codes, scale and zero-point of the rows of x."""
    x = x.float()
    fine = torch.isfinite(x).all(-1, keepdim=True)
    x = torch.where(fine, x, 0.0)
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    scale = ((hi - lo) / 15).clamp(max=65504.0).to(torch.float16)
    back = torch.where(scale > 0, 1.0 / scale.float(), 0.0)
    zero = torch.round(-lo * back).clamp(0, 15)
    code = (torch.round(x * back) + zero).clamp(0, 15)
    scale = torch.where(fine, scale, torch.full_like(scale, math.nan))
    return code.to(torch.int32), scale, zero.to(torch.uint8)


def _places(tok, d):
    """Bytes of a tile that hold a token's codes: K [..][d/2], V [..][d/2], and of its scales and zero-points."""
    j = torch.arange(d // 2, device=DEV)
    k = tok[:, None] * (d // 2) + j
    n, r = 2 * j // (d // 8), 2 * j % (d // 8)              # byte j of a V row: d = 2j and 2j + 1
    h, cc, e = tok // 8, tok % 8 // 2, tok % 2
    word = ((h[:, None] * 8 + n) * 4 + cc[:, None]) * (d // 32) + r // 4
    v = 8 * d + (word * 2 + e[:, None]) * 2 + r % 4 // 2
    return k, v, 16 * d + 2 * tok, 16 * d + 32 + 2 * tok, 16 * d + 64 + tok, 16 * d + 80 + tok


def _append(s, c):
    p, d, cache = c["page"], c["dim"], s["cache"]
    kv, tile = cache.shape[1], cache.shape[3]
    page, tok = s["slots"] // p, s["slots"] % p
    base = ((page[:, None] * kv + torch.arange(kv, device=DEV)) * (p // 16) + tok[:, None] // 16) * tile   # [t][kv]
    k_at, v_at, ks_at, vs_at, kz_at, vz_at = _places(tok % 16, d)
    flat = cache.view(-1)
    two = torch.arange(2, device=DEV)
    out = []
    for x, at, s_at, z_at in ((s["k"], k_at, ks_at, kz_at), (s["v"], v_at, vs_at, vz_at)):
        code, scale, zero = _quantise(x)
        flat[base[:, :, None] + at[:, None]] = (code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8)
        flat[base[:, :, None] + s_at[:, None, None] + two] = scale.view(torch.uint8)
        flat[base + z_at[:, None]] = zero.squeeze(-1)
        byte = flat[base[:, :, None] + at[:, None]]
        code = torch.stack([byte & 15, byte >> 4], -1).view(-1, kv, d).float()
        scale = flat[base[:, :, None] + s_at[:, None, None] + two].contiguous().view(torch.float16).float()
        out.append(((code - flat[base + z_at[:, None]].float()[..., None]) * scale).to(x.dtype))
    return out


def _attention(s, c):
    p, d, kv, h = c["page"], c["dim"], c["kv_heads"], c["q_heads"]
    table, seq, starts, q = s["table"].long(), s["seq"].long(), s["starts"].long(), s["q"]
    n, cols, t, m, group = table.shape[0], table.shape[1], q.shape[0], s["max_q"], h // kv
    length = cols * p
    tiles = length // 16
    raw = s["cache"][table.clamp(min=0)].transpose(1, 2).reshape(n, kv, tiles, 16 * (d + 6))
    scale = raw[..., 16 * d:16 * d + 64].contiguous().view(torch.float16).float().view(n, kv, tiles, 2, 16)
    zero = raw[..., 16 * d + 64:].float().view(n, kv, tiles, 2, 16)
    seen = torch.arange(length, device=DEV)[None] < seq[:, None]                # [n][length]
    ok = seen[:, None, :, None]

    def value(code, which):
        x = (code.float() - zero[..., which, :, None]) * scale[..., which, :, None]
        return torch.where(ok, x.view(n, kv, length, d), 0.0)

    byte = raw[..., :8 * d]
    k = value(torch.stack([byte & 15, byte >> 4], -1).view(n, kv, tiles, 16, d), 0)
    byte = raw[..., 8 * d:16 * d]
    code = torch.stack([byte & 15, byte >> 4], -1).view(n, kv, tiles, 2, 8, 4, d // 32, 2, 4)
    v = value(code.permute(0, 1, 2, 3, 5, 7, 4, 6, 8).reshape(n, kv, tiles, 16, d), 1)
    del raw, byte, code
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


def _sample(s, c):
    x = s["logits"].float()
    n, v = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    warm = s["temp"] > 0
    temp = torch.where(warm, s["temp"], 1.0)
    k = torch.where(warm, torch.where(s["top_k"] > 0, s["top_k"].long(), v), 1)
    top = x.amax(-1, keepdim=True)
    e = torch.where(x == top, 1.0, torch.exp((x - top) * (1.0 / temp)[:, None]))
    e = torch.where((top == -math.inf), 0.0, e)
    # weights are whole numbers of 2^-31: their sums do not depend on an order
    x, order = torch.sort(x, dim=-1, descending=True, stable=True)
    e = e.gather(1, order)
    w = torch.round(e * 2147483648.0).long()
    rank = torch.arange(v, device=DEV)[None]
    w = torch.where(rank < k[:, None], w, 0)
    total = torch.cumsum(w, -1)
    before = (total - w).double()
    keep = before < total[:, -1:].double() * s["top_p"].double()[:, None]
    keep = (keep | (rank == 0)) & ((e >= s["min_p"][:, None]) | (rank == 0))
    w = torch.zeros_like(w).scatter(1, order, torch.where(keep, w, 0))
    total = torch.cumsum(w, -1)
    last = total[:, -1]
    at = torch.minimum((last.double() * s["u"].double()).long(), last - 1)
    token = (total <= at[:, None]).sum(-1)
    none = last == 0
    prob = w.gather(1, token.clamp(max=v - 1)[:, None])[:, 0].double() / torch.where(none, 1, last).double()
    return [torch.where(none, -1, token).to(torch.int32), torch.where(none, 0.0, prob).float()]


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None                                     # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "append":
        out = []
        for x in (s["k"], s["v"]):
            x = x.double()
            lo = torch.minimum(x.min(-1).values, torch.zeros((), dtype=torch.float64, device=DEV))
            hi = torch.maximum(x.max(-1).values, torch.zeros((), dtype=torch.float64, device=DEV))
            step = ((hi - lo) / 15.0).half().double()[..., None]
            zero = torch.round(-lo[..., None] / step)
            out.append(((torch.round(x / step) + zero).clamp(0, 15) - zero) * step)
        return out
    if case["op"] == "sample":
        x = s["logits"].double()
        n, v = x.shape
        probs = torch.zeros(n, dtype=torch.float64, device=DEV)
        for b in range(n):
            t = float(s["temp"][b])
            y = (x[b] - x[b].max()) * (1.0 / t if t > 0 else 1.0)
            order = torch.argsort(y, descending=True, stable=True)
            e = torch.exp(y[order])
            k = int(s["top_k"][b])
            k = 1 if t <= 0 else v if k <= 0 else min(k, v)
            e = e[:k]
            before = torch.cumsum(e, 0) - e
            e = e[(before < e.sum() * float(s["top_p"][b])) & (e >= float(s["min_p"][b]))]
            order = order[:e.numel()]
            by_index = torch.argsort(order)
            e = e[by_index]
            cum = torch.cumsum(e, 0)
            at = int((cum <= cum[-1] * float(s["u"][b])).sum())
            probs[b] = e[min(at, e.numel() - 1)] / cum[-1]
        return [None, probs]
    p, d, kv, h = case["page"], case["dim"], case["kv_heads"], case["q_heads"]
    new, seq = _lengths(case)
    t = sum(new)
    o = torch.zeros(t, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (a, n) in enumerate(zip(new, seq)):
        first, at = at, at + a
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // p)].long()
        for g in range(kv):
            raw = s["cache"][pages, g].reshape(-1, 16 * (d + 6))                # [tiles][bytes]
            kc, vc = raw[:, :8 * d].long().view(-1, 16, d // 2), raw[:, 8 * d:16 * d].long().view(-1, 2, 8, 4, d // 32, 4)
            sc = raw[:, 16 * d:16 * d + 64].contiguous().view(torch.float16).double()
            zc = raw[:, 16 * d + 64:].double()
            key = torch.zeros(raw.shape[0], 16, d, dtype=torch.float64, device=DEV)
            val = torch.zeros_like(key)
            key[..., 0::2], key[..., 1::2] = (kc % 16).double(), (kc // 16).double()
            for tok in range(16):
                two = vc[:, tok // 8, :, tok % 8 // 2, :, 2 * (tok % 2):2 * (tok % 2) + 2]        # [tiles][8][d/32][2]
                val[:, tok] = torch.stack([two % 16, two // 16], -1).reshape(-1, d).double()
            key = ((key - zc[:, :16, None]) * sc[:, :16, None]).view(-1, d)[:n]
            val = ((val - zc[:, 16:, None]) * sc[:, 16:, None]).view(-1, d)[:n]
            pos = torch.arange(n - a, n, device=DEV)[:, None]
            col = torch.arange(n, device=DEV)[None]
            see = (col <= pos) if not case["window"] else (col <= pos) & (col > pos - case["window"])
            for head in range(g * (h // kv), (g + 1) * (h // kv)):
                x = s["q"][first:at, head].double() @ key.T / math.sqrt(d)
                x = x.masked_fill(~see, -math.inf)
                lse[first:at, head] = torch.logsumexp(x, -1)
                o[first:at, head] = torch.softmax(x, -1) @ val
    return [o, lse] if case["lse"] else o
