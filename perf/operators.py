"""What is measured of the attention operators beside the compressors: the per-head norms of queries and
keys with the position rotation, the paged 4-bit K/V cache's writer and reader, and attention over that cache.

``own`` False computes each operator in plain torch operations, True calls libcf.  Both read the same
inputs; a cache is packed here, from the format's definition, for both.

Cache format: a page of P tokens of one K/V head of D channels is one block of P * D * 17 / 16 bytes,
  K codes   [P][D/2]                     low nibble first
  V codes   [P/8][16][8 tokens][D/32]    piece n holds channels n*D/16 .. of each token, low nibble first
  K scales  [P][D/32]                    one byte a group of 32 channels, 2^(byte - 127)
  V scales  [P/8][D/32][8 tokens]
codes are E2M1 (bit 3 the sign, magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6).  The scale's exponent is the least e
with absmax <= 6 * 2^e, held within [-22, 13]; a group with a NaN or an infinity has byte 255 and reads NaN.
"""
import math
import random

import torch

own = False

GROUP = 32
E_MIN, E_MAX = -22, 13
NAN_BYTE = 255
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of a batch of 16: 16 tokens, shared K/V heads; latency is all that counts
        dict(name="norm_step", op="norm", tokens=16, q_heads=32, k_heads=8, dim=128, dtype="bf16", norm="rms", style="half", packed=True, table=32768),
        # one image shard's queries and keys (1024 tokens, 24 heads of 128), out of one packed projection
        dict(name="norm_image", op="norm", tokens=1024, q_heads=24, k_heads=24, dim=128, dtype="bf16", norm="rms", style="interleaved", packed=True, table=4096),
        # a whole video's tokens in fp32, layer norms with biases, 30 heads of 64
        dict(name="norm_video", op="norm", tokens=17550, q_heads=30, k_heads=30, dim=64, dtype="f32", norm="layer", style="interleaved", packed=False, table=17550),
        # one decoding step's K and V of a batch of 61 into their pages, three of them padding
        dict(name="store_step", op="store", tokens=61, heads=8, dim=128, dtype="bf16", page=16, pages=4096, padding=3),
        # an image shard's reconstructions, which receivers hold in fp32, into a cache
        dict(name="store_image", op="store", tokens=1024, heads=24, dim=128, dtype="f32", page=64, pages=64, padding=0),
        # a video's K and V of one layer
        dict(name="store_video", op="store", tokens=17550, heads=30, dim=64, dtype="bf16", page=128, pages=160, padding=0),
        # a single token over one conversation of 4097: the smallest call of a serving loop
        dict(name="attn_token", op="attn", batch=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=16, max_q=1, max_kv=4097, lens="full", causal=True, window=0, mix=0),
        # a serving step of 64 conversations of very different lengths
        dict(name="attn_serve", op="attn", batch=64, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=16, max_q=1, max_kv=32768, lens="ragged", causal=True, window=0, mix=1),
        # three long contexts without shared heads, queries in fp32
        dict(name="attn_long", op="attn", batch=3, q_heads=24, kv_heads=24, dim=128, dtype="f32", page=64, max_q=1, max_kv=65537, lens="full", causal=True, window=0, mix=2),
        # an image shard's 1024 queries over the four shards and the prompt's tokens
        dict(name="attn_image", op="attn", batch=1, q_heads=24, kv_heads=24, dim=128, dtype="bf16", page=64, max_q=1024, max_kv=4608, lens="full", causal=False, window=0, mix=3),
        # a video shard's 2925 queries over the six shards' 17550 tokens
        dict(name="attn_video", op="attn", batch=1, q_heads=30, kv_heads=30, dim=64, dtype="bf16", page=128, max_q=2925, max_kv=17550, lens="full", causal=False, window=0, mix=4),
        # prompts of a serving loop that arrive in chunks behind what is cached, with a window
        dict(name="attn_chunks", op="attn", batch=5, q_heads=32, kv_heads=8, dim=128, dtype="bf16", page=32, max_q=2047, max_kv=9000, lens="ragged", causal=True, window=4096, mix=5),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "store", "attn", "attn"))
    dim, dtype = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "f32"))
    kv_heads = _spread(rng, 1, 30)
    if op == "norm":
        tokens = _spread(rng, 1, 16384)
        return dict(op="norm", tokens=tokens, q_heads=kv_heads * rng.choice((1, 2, 4)) if kv_heads < 9 else kv_heads, k_heads=kv_heads, dim=dim, dtype=dtype,
                    norm=rng.choice(("rms", "layer", "none")), style=rng.choice(("half", "interleaved")), packed=rng.random() < 0.5, table=tokens + rng.randrange(5000))
    page = rng.choice((16, 32, 64, 128))
    if op == "store":
        tokens = _spread(rng, 1, 16384)
        return dict(op="store", tokens=tokens, heads=kv_heads, dim=dim, dtype=dtype, page=page, pages=tokens // page + 1 + rng.randrange(64), padding=rng.randrange(min(tokens, 5)))
    group = rng.choice((1, 1, 3, 4, 8)) if kv_heads < 9 else 1
    max_q = 1 if rng.random() < 0.5 else _spread(rng, 2, 2048)
    batch = _spread(rng, 1, 64) if max_q == 1 else _spread(rng, 1, 6)
    most = min(131072, int(1.5e8 / max_q / (kv_heads * group) / batch) if max_q > 1 else int(1.2e7 / kv_heads / batch))
    causal = rng.random() < 0.6
    return dict(op="attn", batch=batch, q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page, max_q=max_q,
                max_kv=max(max_q, _spread(rng, 1, max(2, most))), lens=rng.choice(("full", "ragged")), causal=causal,
                window=_spread(rng, 1, 8192) if causal and rng.random() < 0.3 else 0, mix=rng.randrange(1 << 20))


def _lengths(case):
    """Query and K/V lengths of each sequence: all full, or mixed, an empty one among them."""
    b, mq, mk = case["batch"], case["max_q"], case["max_kv"]
    if case["lens"] == "full":
        return [mq] * b, [mk] * b
    rng = random.Random(case["mix"])
    qs = [mq if i == 0 else _spread(rng, 1, mq) for i in range(b)]
    ks = [mk if i == 0 else max(qs[i], _spread(rng, 1, mk)) for i in range(b)]
    if b > 2:  # a slot of the batch that holds nothing
        i = rng.randrange(1, b)
        ks[i] = 0
        qs[i] = 1 if mq == 1 else 0
    return qs, ks


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


def work(case):
    esz = DTYPES[case["dtype"]].itemsize
    d = case["dim"]
    if case["op"] == "norm":
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        return {"bytes": rows * d * 2 * esz + case["tokens"] * (d * 4 + 4), "flops": rows * d * 8}
    if case["op"] == "store":
        rows = (case["tokens"] - case["padding"]) * case["heads"]
        return {"bytes": rows * d * (4 * esz + 2 * 17 / 16), "flops": rows * d * 4}
    qs, ks = _lengths(case)
    seen = ks
    if case["causal"] and case["window"]:
        seen = [min(lk, lq + case["window"] - 1) if lq else 0 for lq, lk in zip(qs, ks)]
    elif not all(qs):
        seen = [lk if lq else 0 for lq, lk in zip(qs, ks)]
    return {"bytes": sum(seen) * case["kv_heads"] * d * 17 / 16 + sum(qs) * case["q_heads"] * (d * 2 * esz + 4),
            "flops": 4 * _pairs(case) * case["q_heads"] * d}


# ------------------------------------------------------------------ the cache format, from its definition

def _quantize(x):
    """(codes uint8 in the shape of x, scale bytes uint8 with x's last axis in groups of 32)."""
    g = x.float().unflatten(-1, (-1, GROUP))
    top = g.abs().amax(-1)
    f, e = torch.frexp(top)  # top = f * 2^e, f in [1/2, 1); 6 = 0.75 * 2^3
    e = torch.where(f <= 0.75, e - 3, e - 2).clamp(E_MIN, E_MAX)
    e = torch.where(top > 0, e, E_MIN)
    bad = ~torch.isfinite(top)
    e = torch.where(bad, 0, e)
    y = torch.ldexp(g, -e[..., None]).abs()
    n = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    n = (n | (torch.signbit(g).to(torch.uint8) << 3)).masked_fill(bad[..., None], 0)
    return n.flatten(-2), (e + 127).to(torch.uint8).masked_fill(bad, NAN_BYTE)


def _values(codes, scales, dtype=torch.float32):
    """What codes (..., D) with scale bytes (..., D/32) stand for."""
    c = codes.long()
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=dtype, device=codes.device)[c]
    s = torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), scales.int() - 127)
    s = s.masked_fill(scales == NAN_BYTE, math.nan)
    return (level.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _parts(cache, page, dim):
    """Views of a cache (pages, heads, bytes): K codes, V codes, K scales, V scales."""
    n, h, _ = cache.shape
    a, b = page * dim // 2, page * dim // GROUP
    return (cache[..., :a].view(n, h, page, dim // 2), cache[..., a:2 * a].view(n, h, page // 8, 16, 8, dim // 32),
            cache[..., 2 * a:2 * a + b].view(n, h, page, dim // GROUP), cache[..., 2 * a + b:].view(n, h, page // 8, dim // GROUP, 8))


def _store(cache, page, dim, k, v, slots):
    """Rows k, v (tokens, heads, dim) into the slots of a cache; negative slots take nothing."""
    kc, vc, ks, vs = _parts(cache, page, dim)
    keep = slots >= 0
    s, k, v = slots[keep], k[keep], v[keep]
    p, t = s // page, s % page
    c, e = _quantize(k)
    kc[p, :, t] = c[..., 0::2] | (c[..., 1::2] << 4)
    ks[p, :, t] = e
    c, e = _quantize(v)
    vc[p, :, t // 8, :, t % 8] = (c[..., 0::2] | (c[..., 1::2] << 4)).unflatten(-1, (16, -1))
    vs[p, :, t // 8, :, t % 8] = e


def _load(cache, page, dim, pages, dtype=torch.float32):
    """K and V (len(pages) * page tokens, heads, dim) of these pages."""
    kc, vc, ks, vs = _parts(cache, page, dim)
    h = cache.shape[1]
    kc, ks = kc[pages].transpose(1, 2), ks[pages].transpose(1, 2)
    vc = vc[pages].permute(0, 2, 4, 1, 3, 5).reshape(len(pages), page, h, dim // 2)
    vs = vs[pages].permute(0, 2, 4, 1, 3).reshape(len(pages), page, h, dim // GROUP)

    def rows(c, s):
        return _values(torch.stack((c & 15, c >> 4), -1).flatten(-2), s, dtype).flatten(0, 1)

    return rows(kc, ks), rows(vc, vs)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activation(g, tokens, heads, dim):
    """Token rows as projections give them: each channel with a scale of its own, one in a hundred 20 times as large."""
    scale = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device="cuda"))
    scale = torch.where(torch.rand(heads, dim, generator=g, device="cuda") < 0.01, 20 * scale, scale)
    return torch.randn(tokens, heads, dim, generator=g, device="cuda") * scale


def prepare(case, seed):
    g, dim, dtype = _gen(seed), case["dim"], DTYPES[case["dtype"]]
    if case["op"] == "norm":
        t, hq, hk = case["tokens"], case["q_heads"], case["k_heads"]
        if case["packed"]:  # q, k and v out of one product
            x = _activation(g, t, hq + 2 * hk, dim).to(dtype)
            q, k = x[:, :hq], x[:, hq:hq + hk]
        else:
            q, k = _activation(g, t, hq, dim).to(dtype), _activation(g, t, hk, dim).to(dtype)
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        par = 1 + 0.2 * torch.randn(4, dim, generator=g, device="cuda")
        layer = case["norm"] == "layer"
        return dict(case=case, q=q, k=k, cos=angle.cos().float(), sin=angle.sin().float(),
                    positions=torch.randint(0, case["table"], (t,), generator=g, device="cuda").int(),
                    q_weight=None if case["norm"] == "none" else par[0], k_weight=None if case["norm"] == "none" else par[1],
                    q_bias=par[2] - 1 if layer else None, k_bias=par[3] - 1 if layer else None)
    page = case["page"]
    if case["op"] == "store":
        t, h = case["tokens"], case["heads"]
        slots = torch.randperm(case["pages"] * page, generator=g, device="cuda")[:t] if t < 256 else \
            (torch.randperm(case["pages"], generator=g, device="cuda")[:, None] * page + torch.arange(page, device="cuda")).flatten()[:t]
        slots[t - case["padding"]:] = -1
        return dict(case=case, k=_activation(g, t, h, dim).to(dtype), v=_activation(g, t, h, dim).to(dtype), slots=slots,
                    cache=torch.zeros(case["pages"], h, page * dim * 17 // 16, dtype=torch.uint8, device="cuda"))
    qs, ks = _lengths(case)
    per = [-(-n // page) for n in ks]
    width = max(per + [1])
    pages = sum(per) + 2
    h, hq = case["kv_heads"], case["q_heads"]
    # places that hold no token of a sequence keep what an earlier one left there, whatever its bytes
    cache = torch.randint(0, 256, (pages, h, page * dim * 17 // 16), generator=g, device="cuda", dtype=torch.uint8)
    order = torch.randperm(pages, generator=g, device="cuda")
    table = torch.full((len(ks), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(ks):
        if n:
            mine = order[at:at + per[i]]
            at += per[i]
            table[i, :per[i]] = mine.int()
            slots = (mine[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n]
            k, v = _activation(g, n, h, dim), _activation(g, n, h, dim)
            step = max(1, (1 << 27) // (h * dim))
            for j in range(0, n, step):
                _store(cache, page, dim, k[j:j + step], v[j:j + step], slots[j:j + step])
    total = sum(qs)
    starts = torch.tensor([sum(qs[:i]) for i in range(len(qs) + 1)], dtype=torch.int32, device="cuda")
    return dict(case=case, q=torch.randn(total, hq, dim, generator=g, device="cuda").to(dtype), cache=cache, table=table,
                kv_lens=torch.tensor(ks, dtype=torch.int32, device="cuda"), q_starts=starts, scale=dim ** -0.5)


# ------------------------------------------------------------------ the operators

def _norm_rope(x, weight, bias, cos, sin, norm, style, dtype):
    """cos, sin: (tokens, 1, dim/2), in the type that the sums are held in."""
    x = x.to(cos.dtype)
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    if norm != "none":
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.to(cos.dtype)
    if bias is not None:
        x = x + bias.to(cos.dtype)
    if style == "half":
        a, b = x.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(dtype)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2).to(dtype)


def _norm_plain(s, kind=torch.float32):
    c, p = s["case"], s["positions"].long()
    cos, sin = s["cos"][p][:, None].to(kind), s["sin"][p][:, None].to(kind)
    dtype = s["q"].dtype if kind == torch.float32 else kind
    return [_norm_rope(s[x], s[x + "_weight"], s[x + "_bias"], cos, sin, c["norm"], c["style"], dtype) for x in ("q", "k")]


def _store_plain(s):
    c = s["case"]
    _store(s["cache"], c["page"], c["dim"], s["k"], s["v"], s["slots"])
    kc, vc, ks, vs = _parts(s["cache"], c["page"], c["dim"])
    slots = s["slots"].clamp(min=0)
    p, t = slots // c["page"], slots % c["page"]
    k, v = kc[p, :, t], vc[p, :, t // 8, :, t % 8].flatten(-2)
    none = (s["slots"] < 0)[:, None, None]
    k = _values(torch.stack((k & 15, k >> 4), -1).flatten(-2), ks[p, :, t])
    v = _values(torch.stack((v & 15, v >> 4), -1).flatten(-2), vs[p, :, t // 8, :, t % 8])
    return [x.masked_fill(none, 0).to(s["k"].dtype) for x in (k, v)]


def _attn_plain(s):
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


def run(state):
    s = state
    c = s["case"]
    if own:
        from activation_residual_compression_cf_amd import cf

        if c["op"] == "norm":
            norm = {"none": cf.CF_NORM_NONE, "rms": cf.CF_NORM_RMS, "layer": cf.CF_NORM_LAYER}[c["norm"]]
            rope = cf.CF_ROPE_HALF if c["style"] == "half" else cf.CF_ROPE_INTERLEAVED
            return list(cf.qk_norm_rope(s["q"], s["k"], norm=norm, q_weight=s["q_weight"], k_weight=s["k_weight"], q_bias=s["q_bias"], k_bias=s["k_bias"],
                                        eps=1e-6, rope=rope, cos=s["cos"], sin=s["sin"], positions=s["positions"]))
        cache = cf.KV4Cache(s["cache"], c["page"], c["dim"])
        if c["op"] == "store":
            cf.kv4_append(cache, s["k"], s["v"], s["slots"])
            return list(cf.kv4_read(cache, s["slots"], s["k"].dtype))
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
        return [cf.kv4_attention(s["q"], cache, s["kv_lens"], table=s["table"], q_starts=s["q_starts"], max_q=c["max_q"],
                                 causal=c["causal"], window=c["window"], scale=s["scale"], lse=lse), lse]
    return {"norm": _norm_plain, "store": _store_plain, "attn": _attn_plain}[c["op"]](s)


# ------------------------------------------------------------------ 64 bits

def _exact_norm(s):
    c = s["case"]
    out = []
    at = s["positions"].long()
    # the tables are inputs, so the rotation is by what they hold
    turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]
    for name in ("q", "k"):
        x = s[name].double()
        if c["norm"] == "layer":
            x = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt()
        elif c["norm"] == "rms":
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["dim"] + 1e-6).sqrt()
        if s[name + "_weight"] is not None:
            x = x * s[name + "_weight"].double()
        if s[name + "_bias"] is not None:
            x = x + s[name + "_bias"].double()
        if c["style"] == "half":
            x = x.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_complex(x.contiguous()) * turn
            out.append(torch.view_as_real(z).transpose(-1, -2).flatten(-2))
        else:
            z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous()) * turn
            out.append(torch.view_as_real(z).flatten(-2))
    return out


def _exact_store(s):
    """Each value's nearest level, ties to the level of even index; by distances, not by borders."""
    out = []
    for name in ("k", "v"):
        x = s[name].double().unflatten(-1, (-1, GROUP))
        top = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 6))
        e = torch.where(top > 6 * torch.exp2(e), e + 1, e)
        e = torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
        y = x / torch.exp2(e)
        best, far = torch.zeros_like(y), torch.full_like(y, math.inf)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):
            d = (y.abs() - LEVELS[i]).abs()
            best, far = torch.where(d < far, LEVELS[i], best), torch.minimum(d, far)
        r = (best * torch.sign(y) * torch.exp2(e)).flatten(-2)
        r[s["slots"] < 0] = 0
        out.append(r)
    return out


def _exact_attn(s):
    c = s["case"]
    if _pairs(c) * c["q_heads"] * c["dim"] > 4e11:
        return None
    qs, ks = _lengths(c)
    page, dim, h = c["page"], c["dim"], c["kv_heads"]
    g = c["q_heads"] // h
    out = torch.zeros(*s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for i, (lq, lk) in enumerate(zip(qs, ks)):
        if lq and lk:
            pages = s["table"][i, :-(-lk // page)].long()
            for j in range(h):
                k, v = _load(s["cache"][:, j:j + 1], page, dim, pages, torch.float64)
                k, v = k[:lk, 0], v[:lk, 0]
                for r in range(0, lq, 512):
                    n = min(512, lq - r)
                    x = torch.matmul(s["q"][at + r:at + r + n, j * g:(j + 1) * g].double().reshape(n * g, dim), k.T.contiguous()) * s["scale"]
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
        at += lq
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "store": _exact_store, "attn": _exact_attn}[case["op"]](s)
