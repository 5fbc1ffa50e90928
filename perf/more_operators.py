"""What is measured of the operators around a serving loop's caches: the paged 8-bit K/V cache's writer and
reader, attention over that cache, attention over whole prompts, and the operations on pages (resizing,
forking, compacting, copying).

``own`` False computes each operator in plain torch operations, True calls libcf.  Both read the same
inputs; an 8-bit cache is packed here, from the format's definition, for both.

8-bit cache: a page of P tokens of one K/V head of D channels is one block of 2 P D + max(16, P / 8) bytes,
  K codes   [P][D]
  V codes   [P/8][D][8 tokens]
  K scales  [P/16]        one byte for 16 tokens, 2^(byte - 127)
  V scales  [P/16]
codes are E4M3 (bit 7 the sign, 4 exponent bits of bias 7, magnitudes up to 448, 127 reads NaN).  A scale's
exponent is the least e with max|finite x| <= 448 * 2^e over the 16 tokens, held within [-15, 7]; NaN and infinities
become NaN.  Tokens are appended at the end of sequences.  A call that writes the first of 16 tokens begins them anew;
one that writes others of them keeps the scale or raises it, and rounds what is held to the raised one.

Pages: refs[p] is how many rows of the table hold page p (0: free), table[r] the pages of row r, lens[r] its tokens.
"""
import math
import random

import torch

own = False

BLOCK = 16
E_MIN, E_MAX = -15, 7
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of a batch of 61: a token each, somewhere in its sequence
        dict(name="store8_step", op="store", batch=61, new=1, held=900, lens="ragged", heads=8, dim=128, dtype="bf16", page=16, mix=0),
        # prompts of very different lengths behind what is held already, out of a packed projection
        dict(name="store8_prompts", op="store", batch=5, new=8192, held=700, lens="ragged", heads=24, dim=128, dtype="bf16", page=64, mix=1),
        # a single token over one conversation of 4097: the smallest call of a serving loop
        dict(name="attn8_token", op="attn8", batch=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=16, max_q=1, max_kv=4097, lens="full", causal=True, window=0, mix=0),
        # a serving step of 64 conversations of very different lengths
        dict(name="attn8_serve", op="attn8", batch=64, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=16, max_q=1, max_kv=32768, lens="ragged", causal=True, window=0, mix=1),
        # an image shard's 1024 queries over the four shards and the prompt's tokens, in fp32
        dict(name="attn8_image", op="attn8", batch=1, q_heads=24, kv_heads=24, dim=128, dtype="f32", page=64, max_q=1024, max_kv=4608, lens="full", causal=False, window=0, mix=2),
        # prompts of a serving loop that arrive in chunks behind what is cached, with a window
        dict(name="attn8_chunks", op="attn8", batch=5, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=32, max_q=2047, max_kv=9000, lens="ragged", causal=True, window=4096, mix=3),
        # a handful of short prompts: latency
        dict(name="prompt_short", op="prompt", batch=7, q_heads=32, kv_heads=8, dim=128, dtype="bf16", max_q=333, max_kv=333, lens="ragged", causal=True, window=0, mix=4),
        # long prompts packed behind each other
        dict(name="prompt_long", op="prompt", batch=4, q_heads=32, kv_heads=8, dim=128, dtype="bf16", max_q=16383, max_kv=16383, lens="ragged", causal=True, window=0, mix=5),
        # all tokens of a video, each seeing all: 30 heads of 64
        dict(name="prompt_video", op="prompt", batch=1, q_heads=30, kv_heads=30, dim=64, dtype="bf16", max_q=17550, max_kv=17550, lens="full", causal=False, window=0, mix=6),
        # an image's tokens in fp32
        dict(name="prompt_f32", op="prompt", batch=1, q_heads=24, kv_heads=24, dim=128, dtype="f32", max_q=4096, max_kv=4608, lens="full", causal=False, window=0, mix=7),
        # a step of a search with 8 prompts of 4 beams each: every beam goes on from one of its prompt's, and grows by a token
        dict(name="pages_fork", op="fork", rows=32, beams=4, tokens=700, page=16, layers=2, page_bytes=34944, spare=40, mix=8),
        # a cache of two layers with many pages let go here and there, pushed together
        dict(name="pages_compact", op="compact", rows=64, tokens=9000, page=64, layers=2, page_bytes=139392, spare=3000, mix=9),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("store", "attn8", "attn8", "prompt", "prompt", "fork", "compact"))
    mix = rng.randrange(1 << 20)
    if op in ("fork", "compact"):
        page = rng.choice((16, 32, 64, 128))
        beams = rng.choice((2, 3, 4, 8))
        rows = _spread(rng, 1, 32) * beams
        tokens = _spread(rng, 1, 4000)
        layers = rng.choice((1, 2, 3))
        kind = rng.choice((17, 33))  # 16ths of a byte a channel: a 4-bit cache's, or about an 8-bit one's
        each = rows * (tokens / page + 1) + 1200
        page_bytes = max(16, min(_spread(rng, 1, 30) * page * rng.choice((64, 128)) * kind // 16, int(1e9 / each / layers)) // 16 * 16)
        return dict(op=op, rows=rows, beams=beams, tokens=tokens, page=page, layers=layers, page_bytes=page_bytes,
                    spare=_spread(rng, max(1, rows // 8) if op == "fork" else 1, 1200), mix=mix)
    dim, dtype = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "f32"))
    kv_heads = _spread(rng, 1, 30)
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "store":
        one = rng.random() < 0.5
        batch = _spread(rng, 1, 128) if one else _spread(rng, 1, 6)
        return dict(op=op, batch=batch, new=1 if one else _spread(rng, 2, 20000 // batch), held=_spread(rng, 1, 1000), lens=rng.choice(("full", "ragged")),
                    heads=kv_heads, dim=dim, dtype=dtype, page=page, mix=mix)
    group = rng.choice((1, 1, 3, 4, 8)) if kv_heads < 9 else 1
    causal = rng.random() < 0.6
    base = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, dtype=dtype, lens=rng.choice(("full", "ragged")), causal=causal, mix=mix)
    if op == "attn8":
        max_q = 1 if rng.random() < 0.5 else _spread(rng, 2, 2048)
        batch = _spread(rng, 1, 64) if max_q == 1 else _spread(rng, 1, 6)
        most = min(131072, int(1.5e8 / max_q / (kv_heads * group) / batch) if max_q > 1 else int(1.2e7 / kv_heads / batch))
        base.update(page=page)
    else:
        batch = _spread(rng, 1, 8)
        pairs = (4e9 if dtype == "bf16" else 4e8) / (kv_heads * group) / batch
        max_q = _spread(rng, 1, min(16384, int(math.sqrt(pairs))))
        most = min(32768, int(pairs / max_q))
    max_kv = max(max_q, _spread(rng, 1, max(2, most))) if op == "attn8" or rng.random() < 0.3 else max_q
    base.update(batch=batch, max_q=max_q, max_kv=max_kv, window=_spread(rng, 1, 8192) if causal and rng.random() < 0.3 else 0)
    return base


def _lengths(case):
    """Query and K/V lengths of each sequence: all full, or mixed, an empty one among them."""
    b, mq, mk = case["batch"], case["max_q"], case["max_kv"]
    if case["lens"] == "full":
        return [mq] * b, [mk] * b
    rng = random.Random(case["mix"])
    qs = [mq if i == 0 else _spread(rng, 1, mq) for i in range(b)]
    ks = [mk if i == 0 else qs[i] if case["op"] == "prompt" and mq == mk else max(qs[i], _spread(rng, 1, mk)) for i in range(b)]
    if b > 2:  # a slot of the batch that holds nothing
        i = rng.randrange(1, b)
        ks[i] = 0
        qs[i] = 1 if mq == 1 else 0
    return qs, ks


def _store_lengths(case):
    """New and held tokens of each sequence; one of three or more has none new."""
    rng = random.Random(case["mix"])
    full = case["lens"] == "full"
    new = [case["new"] if full or i == 0 else _spread(rng, 1, case["new"]) for i in range(case["batch"])]
    held = [case["held"] if full else rng.randrange(case["held"] + 1) for _ in new]
    if case["batch"] > 2 and case["new"] > 1:
        new[rng.randrange(1, case["batch"])] = 0
    return new, held


def _pairs(case):
    """(query, key) pairs that the mask leaves, for one head."""
    n = 0
    for lq, lk in zip(*_lengths(case)):
        if not case["causal"]:
            n += lq * lk
            continue
        w = case["window"] or lk
        for i in range(lq):
            n += max(0, min(lk - lq + i + 1, w))
    return n


def _block_bytes(page, dim):
    return 2 * page * dim + max(16, page // 8)


def work(case):
    if case["op"] in ("fork", "compact"):
        rows, held = _rows(case)
        width = max(held) // case["page"] + 2
        pages = sum(-(-n // case["page"]) for n in held) + case["spare"]
        if case["op"] == "fork":
            par = _parents(case)
            moved = sum(1 for r, p in enumerate(par) if p != r and held[p] % case["page"])
            small = 4 * (2 * pages + 2 * rows * width + 3 * rows)
        else:
            moved = _moves(case)
            small = 4 * (2 * pages + 2 * rows * width)
        return {"bytes": small + 2 * moved * case["layers"] * case["page_bytes"], "flops": pages + rows * width}
    esz = DTYPES[case["dtype"]].itemsize
    d = case["dim"]
    if case["op"] == "store":
        new, held = _store_lengths(case)
        rows = sum(new) * case["heads"]
        read = sum(n + (h % BLOCK if n else 0) for n, h in zip(new, held)) * case["heads"]
        return {"bytes": rows * d * 2 * (esz + 1) + read * d * 2 * (1 + esz), "flops": rows * d * 4}
    qs, ks = _lengths(case)
    seen = [lk if lq else 0 for lq, lk in zip(qs, ks)]
    if case["causal"] and case["window"]:
        seen = [min(lk, lq + case["window"] - 1) if lq else 0 for lq, lk in zip(qs, ks)]
    key = d * 2 + 1 / 8 if case["op"] == "attn8" else d * 2 * esz
    return {"bytes": sum(seen) * case["kv_heads"] * key + sum(qs) * case["q_heads"] * (d * 2 * esz + 4),
            "flops": 4 * _pairs(case) * case["q_heads"] * d}


# ------------------------------------------------------------------ the cache format, from its definition

def _two(e, dtype=torch.float32):
    """2^e, exactly."""
    return ((e.int() + 127) << 23).view(torch.float32) if dtype == torch.float32 else ((e.long() + 1023) << 52).view(torch.float64)


def _exponents(top):
    """Least e with top <= 448 * 2^e, within its limits."""
    f, e = torch.frexp(top)  # top = f * 2^e, f in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(f <= 0.875, e - 9, e - 8).clamp(E_MIN, E_MAX)
    return torch.where(top > 0, e, E_MIN)


def _encode(x, e):
    """Codes of x * 2^-e."""
    x = x.float()
    bad = ~torch.isfinite(x)
    a = (x.abs().masked_fill(bad, 0) * _two(-e)).clamp(max=448.0)
    k = torch.frexp(a.clamp(min=2.0 ** -6))[1] - 1  # a in [2^k, 2^(k+1)), or below 2^-6
    n = torch.round(a * _two(3 - k)).int()  # half to even; 16 carries into the next exponent
    code = n + ((k + 6) << 3)  # n >= 8 holds the exponent field's lowest one
    return (code | (torch.signbit(x).int() << 7)).masked_fill(bad, 127).to(torch.uint8)


def _levels(dtype, device):
    """What the 256 codes stand for."""
    c = torch.arange(256, device=device)
    e, m = c >> 3 & 15, (c & 7).to(dtype)
    v = torch.where(e > 0, (1 + m / 8) * _two(e - 7, dtype), m / 8 * 2.0 ** -6)
    v = torch.where(c > 127, -v, v)
    return torch.where((c & 127) == 127, math.nan, v)


def _decode(codes, scales, dtype=torch.float32):
    """What codes stand for; scale bytes broadcast to them."""
    return _levels(dtype, codes.device)[codes.long()] * _two(scales.int() - 127, dtype)


def _parts(cache, page, dim):
    """Views of a cache (pages, heads, bytes): K codes, V codes, K scales, V scales."""
    n, h, _ = cache.shape
    a, b = page * dim, page // BLOCK
    return (cache[..., :a].view(n, h, page, dim), cache[..., a:2 * a].view(n, h, page // 8, dim, 8),
            cache[..., 2 * a:2 * a + b], cache[..., 2 * a + b:2 * a + 2 * b])


def _append(cache, page, dim, k, v, slots):
    """Rows k, v (tokens, heads, dim) into slots, which are the ends of sequences; negative slots take nothing."""
    kc, vc, ks, vs = _parts(cache, page, dim)
    n, h = cache.shape[:2]
    per, dev = page // BLOCK, cache.device
    keep = (slots >= 0).nonzero()[:, 0]
    slot, k, v = slots[keep], k[keep].float(), v[keep].float()
    # the blocks that take something, and which of them each token is of
    block, mine = torch.unique(slot // BLOCK, return_inverse=True)
    anew = torch.zeros(len(block), dtype=torch.int32, device=dev).index_add_(0, mine, (slot % BLOCK == 0).int()) > 0
    bp, bt, p, t = block // per, block % per, slot // page, slot % page
    for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
        blocks = codes.view(n, h, per, BLOCK, dim) if codes is kc else codes.view(n, h, per, 2, dim, 8).transpose(-1, -2)
        held = blocks[bp, :, bt]
        top = torch.where(torch.isfinite(x), x.abs(), 0).amax(-1)
        e = _exponents(torch.zeros(len(block), h, device=dev).scatter_reduce_(0, mine[:, None].expand_as(top), top, "amax"))
        old = scales[bp, :, bt].int().sub(127).clamp(E_MIN, E_MAX)
        e = torch.where(anew[:, None], e, torch.maximum(e, old))
        wide = (...,) + (None,) * (held.dim() - 2)
        blocks[bp, :, bt] = torch.where((old < e)[wide], _encode(_decode(held, (old + 127)[wide]), e[wide]), held)
        scales[bp, :, bt] = (e + 127).to(torch.uint8)
        new = _encode(x, e[mine][..., None])
        if codes is kc:
            codes[p, :, t] = new
        else:
            codes[p, :, t // 8, :, t % 8] = new


def _read(cache, page, dim, slots, dtype=torch.float32):
    kc, vc, ks, vs = _parts(cache, page, dim)
    slot = slots.clamp(min=0)
    p, t = slot // page, slot % page
    k = _decode(kc[p, :, t], ks[p, :, t // BLOCK][..., None], dtype)
    v = _decode(vc[p, :, t // 8, :, t % 8], vs[p, :, t // BLOCK][..., None], dtype)
    none = (slots < 0)[:, None, None]
    return k.masked_fill(none, 0), v.masked_fill(none, 0)


def _load(cache, page, dim, pages, dtype=torch.float32):
    """K and V (len(pages) * page tokens, heads, dim) of these pages."""
    kc, vc, ks, vs = _parts(cache, page, dim)
    n, h, per = len(pages), cache.shape[1], page // BLOCK
    k = _decode(kc[pages].view(n, h, per, BLOCK, dim), ks[pages][..., None, None], dtype)
    v = _decode(vc[pages].view(n, h, per, 2, dim, 8), vs[pages][..., None, None, None], dtype).transpose(-1, -2)
    return k.flatten(2, 3).transpose(1, 2).flatten(0, 1), v.flatten(2, 4).transpose(1, 2).flatten(0, 1)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activation(g, tokens, heads, dim):
    """Token rows as projections give them: each channel with a scale of its own, one in a hundred 20 times as large."""
    scale = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
    scale = torch.where(torch.rand(heads, dim, generator=g, device="cuda") < 0.01, 20 * scale, scale)
    return torch.randn(tokens, heads, dim, generator=g, device="cuda") * scale


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(lens):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def _paged(g, lens, page, heads, dim):
    """A cache of random bytes with a table of pages in any order for sequences of these lengths."""
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 2
    cache = torch.randint(0, 256, (pages, heads, _block_bytes(page, dim)), generator=g, device="cuda", dtype=torch.uint8)
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((len(lens), max(per + [1])), -1, dtype=torch.int32, device="cuda")
    slots, at = [], 0
    for i, n in enumerate(lens):
        mine = order[at:at + per[i]]
        at += per[i]
        table[i, :per[i]] = mine.int()
        slots.append((mine[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n])
    return cache, table, slots


def _fill(g, cache, page, dim, slots):
    step = max(BLOCK, (1 << 25) // (cache.shape[1] * dim) // BLOCK * BLOCK)
    for s in slots:
        k, v = _activation(g, len(s), cache.shape[1], dim), _activation(g, len(s), cache.shape[1], dim)
        for j in range(0, len(s), step):
            _append(cache, page, dim, k[j:j + step], v[j:j + step], s[j:j + step])


def _rows(case):
    """Rows of the table and the tokens of each; beams of one prompt have as many."""
    rng = random.Random(case["mix"])
    if case["op"] == "fork":
        held = [n for n in (_spread(rng, 1, case["tokens"]) for _ in range(case["rows"] // case["beams"])) for _ in range(case["beams"])]
    else:
        held = [case["tokens"] if i == 0 else _spread(rng, 1, case["tokens"]) for i in range(case["rows"])]
    return len(held), held


def _parents(case):
    rng = random.Random(case["mix"] + 1)
    b = case["beams"]
    return [r // b * b + rng.randrange(b) for r in range(case["rows"])]


def _order(case, pages):
    """The pages in the order in which rows took them."""
    order = list(range(pages))
    random.Random(case["mix"] + 2).shuffle(order)
    return order


def _pages_state(case):
    """refs, table and lens, as lists: beams share all their prompt's whole pages but the last one or two."""
    rows, held = _rows(case)
    page = case["page"]
    per = [-(-n // page) for n in held]
    width = max(held) // page + 2
    pages = sum(per) + case["spare"]
    order = _order(case, pages)
    refs, table, at = [0] * pages, [[-1] * width for _ in range(rows)], 0
    for r in range(rows):
        lead = r // case["beams"] * case["beams"] if case["op"] == "fork" else r
        for j in range(per[r]):
            if lead != r and j < held[r] // page - 1:
                table[r][j] = table[lead][j]
            else:
                table[r][j] = order[at]
                at += 1
            refs[table[r][j]] += 1
    return refs, table, held


def _moves(case):
    refs = _pages_state(case)[0]
    live = sum(1 for x in refs if x)
    return sum(1 for x in refs[:live] if not x)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("fork", "compact"):
        refs, table, lens = _pages_state(case)
        s = dict(case=case, refs=_ints(refs), table=_ints(table), lens=_ints(lens),
                 data=torch.randint(0, 256, (case["layers"], len(refs), case["page_bytes"]), generator=g, device="cuda", dtype=torch.uint8))
        if case["op"] == "fork":
            par = _parents(case)
            s.update(parents=_ints(par), want=_ints([lens[p] + 1 for p in par]))
        return s
    dim, dtype = case["dim"], DTYPES[case["dtype"]]
    if case["op"] == "store":
        new, held = _store_lengths(case)
        both = [a + b for a, b in zip(new, held)]
        h, page = case["heads"], case["page"]
        cache, table, slots = _paged(g, both, page, h, dim)
        _fill(g, cache, page, dim, [x[:b] for x, b in zip(slots, held)])
        t = sum(new)
        x = _activation(g, t, 3 * h, dim).to(dtype)  # q, k and v out of one product
        # the new tokens, and those before them whose scale they share
        back = [x[b // BLOCK * BLOCK:] if n else x[:0] for x, n, b in zip(slots, new, held)]
        return dict(case=case, k=x[:, h:2 * h], v=x[:, 2 * h:], cache=cache, table=table, kv_lens=_ints(both), starts=_starts(new),
                    slots=torch.cat([x[b:] for x, b in zip(slots, held)]), back=torch.cat(back))
    qs, ks = _lengths(case)
    h, hq, total = case["kv_heads"], case["q_heads"], sum(qs)
    s = dict(case=case, q=torch.randn(total, hq, dim, generator=g, device="cuda").to(dtype), q_starts=_starts(qs), scale=dim ** -0.5)
    if case["op"] == "attn8":
        cache, table, slots = _paged(g, ks, case["page"], h, dim)
        _fill(g, cache, case["page"], dim, slots)
        s.update(cache=cache, table=table, kv_lens=_ints(ks))
    else:
        x = _activation(g, sum(ks), 2 * h, dim).to(dtype)  # k and v lie beside each other
        s.update(k=x[:, :h], v=x[:, h:], k_starts=_starts(ks))
    return s


# ------------------------------------------------------------------ the operators

def _store_plain(s):
    c = s["case"]
    _append(s["cache"], c["page"], c["dim"], s["k"], s["v"], s["slots"])
    return [x.to(s["k"].dtype) for x in _read(s["cache"], c["page"], c["dim"], s["back"])]


def _hidden(c, lq, lk, r, n, device):
    """(n, lk): the keys that queries r .. r + n - 1 of lq do not see."""
    at = (lk - lq + r + torch.arange(n, device=device))[:, None]
    key = torch.arange(lk, device=device)[None]
    hidden = key > at
    return hidden | (key <= at - c["window"]) if c["window"] else hidden


def _prompt_plain(s):
    c = s["case"]
    h, dim, g = c["kv_heads"], c["dim"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros_like(s["q"])
    lse = torch.full(s["q"].shape[:2], -math.inf, device=s["q"].device)
    a = b = 0
    for lq, lk in zip(*_lengths(c)):
        if lq and lk:
            k = s["k"][b:b + lk].float().permute(1, 2, 0).contiguous()
            v = s["v"][b:b + lk].float().transpose(0, 1).contiguous()
            n = max(1, min(lq, (1 << 30) // (c["q_heads"] * lk)))
            for r in range(0, lq, n):
                m = min(n, lq - r)
                q = s["q"][a + r:a + r + m].float().view(m, h, g, dim).permute(1, 0, 2, 3).reshape(h, m * g, dim)
                x = torch.bmm(q, k).mul_(s["scale"])
                if c["causal"]:
                    x.view(h, m, g, lk).masked_fill_(_hidden(c, lq, lk, r, m, x.device)[None, :, None], -math.inf)
                top = x.amax(-1, keepdim=True)
                p = x.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
                z = p.sum(-1, keepdim=True)
                o = torch.bmm(p, v) / z.masked_fill(z == 0, 1)
                out[a + r:a + r + m] = o.view(h, m, g, dim).permute(1, 0, 2, 3).reshape(m, h * g, dim).to(out.dtype)
                lse[a + r:a + r + m] = (top + z.log())[..., 0].view(h, m, g).permute(1, 0, 2).reshape(m, h * g)
        a, b = a + lq, b + lk
    return [out, lse]


def _attn8_plain(s):
    c = s["case"]
    b, hq, h, dim, page = c["batch"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    total = s["q"].shape[0]
    width = s["table"].shape[1] * page
    dev = s["q"].device
    k, v = _load(s["cache"], page, dim, s["table"].clamp(min=0).long().flatten())
    lens = s["kv_lens"].long()[:, None]
    past = torch.arange(width, device=dev)[None] >= lens
    k, v = k.view(b, width, h, dim), v.view(b, width, h, dim).masked_fill(past[..., None, None], 0)
    # queries padded to (sequence, place in the sequence)
    most = c["max_q"]
    starts = s["q_starts"].long()
    row = torch.arange(total, device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    place = row - starts[seq]
    q = torch.zeros(b, most, hq, dim, device=dev)
    q[seq, place] = s["q"].float()
    g = hq // h
    q = q.view(b, most, h, g, dim).permute(0, 2, 3, 1, 4).reshape(b * h, g * most, dim)
    kt = k.permute(0, 2, 3, 1).reshape(b * h, dim, width).contiguous()
    score = torch.bmm(q, kt).mul_(s["scale"]).view(b, h, g, most, width)
    key = torch.arange(width, device=dev)
    hidden = past[:, None, :].expand(b, most, width)
    if c["causal"]:
        at = lens + torch.arange(most, device=dev)[None] - (starts[1:] - starts[:-1])[:, None]
        hidden = hidden | (key > at[..., None])
        if c["window"]:
            hidden = hidden | (key <= at[..., None] - c["window"])
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top.masked_fill(top == -math.inf, 0)).exp_()
    total_p = score.sum(-1, keepdim=True)
    vv = v.permute(0, 2, 1, 3).reshape(b * h, width, dim).contiguous()
    out = torch.bmm(score.view(b * h, g * most, width), vv).view(b, h, g, most, dim) / total_p.masked_fill(total_p == 0, 1)
    lse = (top + total_p.log())[..., 0].masked_fill(total_p[..., 0] == 0, -math.inf)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, most, hq, dim)[seq, place].to(s["q"].dtype)
    return [out, lse.permute(0, 3, 1, 2).reshape(b, most, hq)[seq, place].contiguous()]


def _holders(refs, table, count, sign):
    """Adds sign for each of the first `count` pages of each row."""
    col = torch.arange(table.shape[1], device=table.device)
    on = (col < count[:, None]) & (table >= 0) & (table < len(refs))
    refs.index_add_(0, table.clamp(0, len(refs) - 1).flatten().long(), (on * sign).int().flatten())


def _free_list(refs):
    """The free pages in order, -1 behind them, and how many there are."""
    free = refs == 0
    n = len(refs)
    at = torch.where(free, free.cumsum(0) - 1, n)
    every = torch.arange(n, device=refs.device)
    return torch.full((n + 1,), -1, device=refs.device).scatter_(0, at, torch.where(free, every, -1))[:n], free.sum()


def _fork_plain(s):
    c, page = s["case"], s["case"]["page"]
    refs, table, lens = s["refs"].clone(), s["table"], s["lens"]
    rows, width = table.shape
    dev = refs.device
    row, col = torch.arange(rows, device=dev), torch.arange(width, device=dev)
    par = s["parents"].long()
    on = (par >= 0) & (par < rows)
    q = par.clamp(0, rows - 1)
    size = torch.where(on, lens[q], 0).long()
    count = (size + page - 1) // page
    new = torch.where(col < count[:, None], table[q], -1)
    # of the rows that go on from one with a part of a page, itself or else the first keeps it
    first = torch.full((rows,), rows, device=dev).scatter_reduce(0, q, torch.where(on, torch.where(row == par, -1, row), rows), "amin")
    keeps = torch.where(row == par, -1, row) == first[q]
    last = (count - 1).clamp(min=0)
    old = new[row, last]
    fresh = on & (size % page != 0) & ~keeps & (old >= 0) & (old < len(refs))
    _holders(refs, table, (lens + page - 1) // page, -1)
    _holders(refs, new, torch.where(fresh, last, count), 1)
    free, many = _free_list(refs)
    at = fresh.cumsum(0) - 1
    gets = fresh & (at < many)
    page_of = torch.where(gets, free[at.clamp(0, len(free) - 1)], -1)
    refs.index_add_(0, page_of.clamp(min=0), gets.int())
    new[row, last] = torch.where(fresh, page_of, old.long()).int()
    size = torch.where(fresh & ~gets, size // page * page, size).int()
    src, dst = torch.where(gets, old, -1), page_of.int()
    missing = [(fresh & ~gets).sum().int().view(1)]
    # each goes on by a token
    want = s["want"].long()
    grow = ((want + page - 1) // page - (size + page - 1) // page).clamp(min=0)
    have = (size + page - 1) // page
    _holders(refs, new, have, -1)
    keep = torch.minimum(have, (want + page - 1) // page)
    new = torch.where((col >= keep[:, None]), -1, new)
    _holders(refs, new, keep, 1)
    free, many = _free_list(refs)
    end = grow.cumsum(0)
    ok = (grow == 0) | (end <= many) & (want <= width * page)
    rank = (end - grow)[:, None] + col - have[:, None]
    takes = ok[:, None] & (col >= have[:, None]) & (rank < end[:, None])
    got = free[rank.clamp(0, len(free) - 1)]
    new = torch.where(takes, got, new).int()
    refs.index_add_(0, torch.where(takes, got, 0).flatten(), takes.int().flatten())
    size = torch.where(ok, want, size).int()
    missing.append((~ok).sum().int().view(1))
    # and the data
    take = src >= 0
    s["data"][:, dst[take].long()] = s["data"][:, src[take].long()]
    return [refs, new, size, src, dst, torch.cat(missing), s["data"]]


def _compact_plain(s):
    refs, table = s["refs"], s["table"]
    n = len(refs)
    dev = refs.device
    every = torch.arange(n, device=dev)
    used = refs != 0
    live = used.sum()
    hole, mover = ~used & (every < live), used & (every >= live)
    cap = n // 2
    src = torch.full((n + 1,), -1, device=dev).scatter_(0, torch.where(mover, mover.cumsum(0) - 1, n), every)[:cap]
    dst = torch.full((n + 1,), -1, device=dev).scatter_(0, torch.where(hole, hole.cumsum(0) - 1, n), every)[:cap]
    take = src >= 0
    to = every.clone()
    to[src[take]] = dst[take]
    ok = (table >= 0) & (table < n)
    new = torch.where(ok, to[table.clamp(0, n - 1).long()].int(), table)
    out = torch.zeros_like(refs).index_add_(0, to, refs)
    s["data"][:, dst[take]] = s["data"][:, src[take]]
    return [out, new, s["lens"].clone(), src.int(), dst.int(), hole.sum().int().view(1), s["data"]]


def run(state):
    s = state
    c = s["case"]
    if own:
        from activation_residual_compression_cf_amd import cf

        if c["op"] in ("fork", "compact"):
            have = cf.PageTable(s["refs"], s["table"], s["lens"], c["page"])
            if c["op"] == "fork":
                new, src, dst, short = cf.pages_fork(have, s["parents"])
                new, none = cf.pages_resize(new, s["want"], out=new)
                cf.pages_copy(s["data"], src, dst)
                return [new.refs, new.table, new.lens, src, dst, torch.cat((short, none)), s["data"]]
            new, src, dst, count = cf.pages_compact(have)
            cf.pages_copy(s["data"], src, dst, count)
            return [new.refs, new.table, new.lens, src, dst, count, s["data"]]
        if c["op"] == "prompt":
            lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
            return [cf.attention(s["q"], s["k"], s["v"], q_starts=s["q_starts"], k_starts=s["k_starts"], max_q=c["max_q"], causal=c["causal"], window=c["window"],
                                 scale=s["scale"], lse=lse), lse]
        cache = cf.KV8Cache(s["cache"], c["page"], c["dim"])
        if c["op"] == "store":
            cf.kv8_append(cache, s["k"], s["v"], s["kv_lens"], table=s["table"], starts=s["starts"])
            return list(cf.kv8_read(cache, s["back"], s["k"].dtype))
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
        return [cf.kv8_attention(s["q"], cache, s["kv_lens"], table=s["table"], q_starts=s["q_starts"], max_q=c["max_q"],
                                 causal=c["causal"], window=c["window"], scale=s["scale"], lse=lse), lse]
    return {"store": _store_plain, "attn8": _attn8_plain, "prompt": _prompt_plain, "fork": _fork_plain, "compact": _compact_plain}[c["op"]](s)


# ------------------------------------------------------------------ 64 bits

def _nearest(x, e):
    """Each value of x * 2^-e taken to the nearest level, ties to the level of even index; by distances to its two neighbours."""
    levels = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (k - 10) for k in range(1, 16) for m in range(8)][:-1], dtype=torch.float64, device=x.device)
    unit = torch.tensor([2.0 ** i for i in range(E_MIN, E_MAX + 1)], dtype=torch.float64, device=x.device)[(e - E_MIN).long()]
    y = (x.abs() / unit).clamp(max=448.0).nan_to_num(0.0)
    hi = torch.searchsorted(levels, y).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    a, b = y - levels[lo], levels[hi] - y
    best = torch.where((a < b) | (a == b) & (lo % 2 == 0), levels[lo], levels[hi])
    return torch.where(torch.isfinite(x), torch.copysign(best, x) * unit, math.nan)


def _least(top):
    e = torch.full_like(top, E_MIN)
    for i in range(E_MIN, E_MAX):
        e = torch.where(top > 448 * 2.0 ** i, i + 1.0, e)
    return e


def _exact_store(s):
    c = s["case"]
    page, dim, h = c["page"], c["dim"], c["heads"]
    new, held = _store_lengths(c)
    out, at = ([], []), 0
    for i, (n, b) in enumerate(zip(new, held)):
        if n:
            f = b // BLOCK * BLOCK
            pos = torch.arange(f, b, device="cuda")
            slot = s["table"][i].long()[pos // page] * page + pos % page
            for y, x, scales, old in zip(out, (s["k"], s["v"]), _parts(s["cache"], page, dim)[2:], _read(s["cache"], page, dim, slot, torch.float64)):
                z = torch.cat((old, x[at:at + n].double()))
                blocks = -(-len(z) // BLOCK)
                z = torch.cat((z, z.new_zeros(blocks * BLOCK - len(z), h, dim))).view(blocks, BLOCK, h, dim)
                fresh = z.clone()
                fresh[0, :b - f] = 0  # what is held counts by its scale
                e = _least(torch.where(torch.isfinite(fresh), fresh.abs(), 0).amax((1, 3)))
                if b > f:
                    p = int(s["table"][i, f // page])
                    was = scales[p, :, f % page // BLOCK].double() - 127
                    e[0] = torch.maximum(e[0], was)
                r = _nearest(z, e[:, None, :, None])
                y.append(r.view(-1, h, dim)[:b - f + n])
        at += n
    return [torch.cat(x) for x in out]


def _exact_attn(s):
    c = s["case"]
    if _pairs(c) * c["q_heads"] * c["dim"] > 1.2e12:
        return None
    qs, ks = _lengths(c)
    dim, h = c["dim"], c["kv_heads"]
    g = c["q_heads"] // h
    out = torch.zeros(*s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = key0 = 0
    for i, (lq, lk) in enumerate(zip(qs, ks)):
        if lq and lk:
            for j in range(h):
                if c["op"] == "attn8":
                    k, v = _load(s["cache"][:, j:j + 1], c["page"], dim, s["table"][i, :-(-lk // c["page"])].long(), torch.float64)
                    k, v = k[:lk, 0], v[:lk, 0]
                else:
                    k, v = s["k"][key0:key0 + lk, j].double(), s["v"][key0:key0 + lk, j].double()
                k = k.T.contiguous()
                for r in range(0, lq, 1024):
                    n = min(1024, lq - r)
                    x = torch.matmul(s["q"][at + r:at + r + n, j * g:(j + 1) * g].double().reshape(n * g, dim), k) * s["scale"]
                    if c["causal"]:
                        pos = (lk - lq + r + torch.arange(n, device="cuda")).repeat_interleave(g)[:, None]
                        key = torch.arange(lk, device="cuda")[None]
                        see = key <= pos
                        if c["window"]:
                            see &= key > pos - c["window"]
                        x = torch.where(see, x, -math.inf)
                    z = torch.logsumexp(x, -1)
                    p = torch.exp(x - torch.where(z == -math.inf, 0, z)[:, None])
                    out[at + r:at + r + n, j * g:(j + 1) * g] = torch.matmul(p, v).view(n, g, dim)
                    lse[at + r:at + r + n, j * g:(j + 1) * g] = z.view(n, g)
        at, key0 = at + lq, key0 + lk
    return [out, lse]


def _exact_fork(s):
    """Row by row, with a list of the free pages."""
    c, page = s["case"], s["case"]["page"]
    refs, table, lens = _pages_state(c)
    par, width = _parents(c), len(table[0])
    rows = len(par)
    holds = [table[r][:-(-lens[r] // page)] for r in range(rows)]
    keeper = {}
    for r in list(reversed(range(rows))) + [r for r in range(rows) if par[r] == r]:
        keeper[par[r]] = r
    now, fresh = [], []
    for r in range(rows):
        new = list(holds[par[r]])
        if lens[par[r]] % page and keeper[par[r]] != r:
            fresh.append((r, new.pop()))
        now.append(new)
    count = [0] * len(refs)
    for new in now:
        for p in new:
            count[p] += 1
    src, dst, size, missing = [-1] * rows, [-1] * rows, [lens[p] for p in par], [0, 0]
    free = [p for p, x in enumerate(count) if not x]
    for r, p in fresh:
        if not free:
            missing[0] += 1
            now[r].append(-1)
            size[r] = size[r] // page * page
            continue
        src[r], dst[r] = p, free.pop(0)
        count[dst[r]] = 1
        now[r].append(dst[r])
    full = False
    for r in range(rows):
        now[r] = now[r][:-(-size[r] // page)]
        w = lens[par[r]] + 1
        need = -(-w // page) - len(now[r])
        full = full or need > len(free)
        if need and (full or w > width * page):
            missing[1] += 1
            continue
        for _ in range(need):
            now[r].append(free.pop(0))
            count[now[r][-1]] = 1
        size[r] = w
    data = s["data"].clone()
    for a, b in zip(src, dst):
        if a >= 0:
            data[:, b] = s["data"][:, a]
    return [_ints(count), _ints([x + [-1] * (width - len(x)) for x in now]), _ints(size), _ints(src), _ints(dst), _ints(missing), data]


def _exact_compact(s):
    refs, table, lens = _pages_state(s["case"])
    n = len(refs)
    used = [p for p in range(n) if refs[p]]
    free = [p for p in range(n) if not refs[p]]
    pairs = [(a, b) for a, b in zip([p for p in used if p >= len(used)], free)]
    to = dict(pairs)
    out = [0] * n
    for p in used:
        out[to.get(p, p)] = refs[p]
    data = s["data"].clone()
    for a, b in pairs:
        data[:, b] = s["data"][:, a]
    pad = [-1] * (n // 2 - len(pairs))
    return [_ints(out), _ints([[to.get(p, p) for p in row] for row in table]), _ints(lens), _ints([a for a, _ in pairs] + pad), _ints([b for _, b in pairs] + pad),
            _ints([len(pairs)]), data]


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "attn8": _exact_attn, "prompt": _exact_attn, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)
