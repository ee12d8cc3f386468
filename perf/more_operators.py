"""The operators of a 4-bit paged KV cache, and what a round answers with: what is measured.

Four operators, beside those of the 8-bit cache and the verification of drafts:

  append     norms of queries and keys per head with the position rotation, keys and values
             written to the cache in 4 bits; then the new tokens read back, as the values that
             the cache holds for them
  read       tokens of the cache by their slots, as FP16 rows
  attention  attention of a round's rows over that cache
  logprobs   log probabilities of given tokens, with entropy and the likeliest alternatives

The cache holds pages of 64 tokens.  Of every token and KV head, each 16 dimensions are one group:
E2M1 codes with an E4M3 scale; a value is code * scale * unit, the unit a float32 number of the
head.  With G = D / 64, token 16 t + c and dimension 16 (G g + i) + e (t, g < 4; c, e < 16; i < G):

  keys    [2 G, 64, 16] bytes: the n = t G + i'th eight bytes of the lane 16 g + c hold the codes
          e = 0 .. 15 (the lower four bits first): row n // 2, lane, bytes 8 (n % 2) on;
  scales  [64, 4 G]: lane 16 g + c, place n.

Token 16 t + 4 g + r and dimension 16 (G a + i) + 4 j + b (t, g, r, a, j, b < 4; i < G):

  values  [2 G, 64, 16] bytes: lane 16 g + 4 a + b has 32 G bytes, 16 of every row; their half
          bytes are the codes of (t, r, i, j) in this order;
  scales  [G, 16, 16]: row i, lane 4 g + a, place 4 t + r.

Sizes: 40 query and 8 key/value heads of 128 dimensions make the 7168 output channels of the
QKV projection that the benchmark times (10 and 2 heads on one of four tensor-parallel shards),
8 rows are its verify block, 256 rows its largest prefill block, 151936 its vocabulary.
"""
import math

import torch

own = False

PAGE = 64
UNIT = 0.125
EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _attn(name, requests, rows, tokens, q_heads=40, kv_heads=8, dim=128, window=0, ragged=False):
    return dict(name=name, op="attention", requests=requests, rows=rows, tokens=tokens,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, window=window, ragged=ragged)


def _append(name, requests, rows, tokens, q_heads=40, kv_heads=8, dim=128, rot=128,
            interleaved=False, norm=True, pad=0):
    return dict(name=name, op="append", requests=requests, rows=rows, tokens=tokens,
                q_heads=q_heads, kv_heads=kv_heads, dim=dim, rot=rot, interleaved=interleaved,
                norm=norm, pad=pad)


def _read(name, requests, rows, kv_heads=8, dim=128, pad=0):
    return dict(name=name, op="read", requests=requests, rows=rows, tokens=0, kv_heads=kv_heads, dim=dim, pad=pad)


def _logprobs(name, rows, vocab, top, temperature):
    return dict(name=name, op="logprobs", rows=rows, vocab=vocab, top=top, temperature=temperature)


def listed():
    return [
        # plain decoding, one token of one request
        _append("append 1 row", 1, 1, 1777),
        # prompt blocks of four requests
        _append("append 4x256 rows", 4, 256, 1000),
        # a short prefix, taken over by another request
        _read("read 777 tokens", 1, 777),
        # a long document's keys and values, for a pass that wants them whole
        _read("read 4x8k tokens", 4, 8192),
        # the first tokens of an answer: latency alone
        _attn("attention 1 row 300", 1, 1, 300),
        # the verify block over a chat's history
        _attn("attention 8 rows 5001", 1, 8, 5001),
        # the verify block at the longest context: the cache's bytes are all that counts
        _attn("attention 8 rows 244k", 1, 8, 244608),
        # many requests on one of four tensor-parallel shards, lengths and rows ragged
        _attn("attention 64 ragged", 64, 8, 12000, 10, 2, 128, 0, True),
        # a prompt block of 256 rows late in a long prompt: matrix work
        _attn("attention 256 rows 16k", 1, 256, 16500),
        # the token just sampled, with the most alternatives that servers offer
        _logprobs("logprobs 1 row top 20", 1, 151936, 20, 1.0),
        # a verify block's rows
        _logprobs("logprobs 8 rows top 5", 8, 151936, 5, 0.8),
        # a prompt block: every token's log probability
        _logprobs("logprobs 256 rows top 20", 256, 151936, 20, 1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, groups):
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice(groups)
    dim = rng.choice([64, 128, 128, 256])
    while kv_heads * group * dim > 5120:
        group = max(1, group // 2)
        kv_heads = max(1, kv_heads // 2) if group == 1 else kv_heads
    return kv_heads, group, dim


def draw(rng):
    kind = rng.choice(["append", "append", "read", "attention", "attention", "attention", "logprobs", "logprobs"])
    if kind == "append":
        kv_heads, group, dim = _heads(rng, [1, 2, 4, 5, 8])
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        requests = _log_int(rng, 1, 32)
        rows = min(_log_int(rng, 1, 256), max(1, 1024 // requests))
        c = _append("", requests, rows, _log_int(rng, 1, 200000), kv_heads * group, kv_heads, dim,
                    rot, rng.random() < 0.3, rng.random() < 0.8, rng.choice([0, 0, 3]))
    elif kind == "read":
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        requests = _log_int(rng, 1, 32)
        most = 32768 * 1024 // (requests * kv_heads * dim)
        c = _read("", requests, _log_int(rng, 1, max(2, min(32768, most))), kv_heads, dim, rng.choice([0, 0, 5]))
    elif kind == "attention":
        kv_heads, group, dim = _heads(rng, [1, 2, 4, 5, 8, 16])
        requests = _log_int(rng, 1, 64)
        rows = rng.choice([1, 1, 4, 8, 8, rng.randint(2, 8), _log_int(rng, 9, 256)])
        room = 244000 * 8 * 128 // (requests * kv_heads * dim)
        room = min(room, 160_000_000 // (requests * kv_heads * group * rows))
        tokens = _log_int(rng, 30, max(31, min(244000, room)))
        if rows > 8:
            tokens = max(rows, min(tokens, 16000 * 256 * 5120 // (rows * requests * kv_heads * group * dim)))
        window = rng.choice([0, 0, 0, rng.randint(1, max(2, tokens))])
        c = _attn("", requests, rows, tokens, kv_heads * group, kv_heads, dim, window, requests > 1)
    else:
        vocab = _log_int(rng, 1000, 151936)
        c = _logprobs("", _log_int(rng, 1, 256), vocab, rng.choice([0, 1, 5, 20, 20, rng.randint(2, 32)]),
                      rng.choice([0.3, 0.7, 1.0, 1.3]))
    del c["name"]
    return c


# ---------------------------------------------------------------- lengths (of the case alone)

def _lengths(c):
    """(rows, tokens before them) of each request."""
    n, rows, tokens = c["requests"], c["rows"], c["tokens"]
    got = []
    for i in range(n):
        part = 1.0 if i == 0 else (i * 0.6180339887498949) % 1.0
        r = rows if i == 0 or not c.get("ragged") else (i * 5 + 3) % (rows + 1)
        total = max(r, int(tokens * part), 1) if c["op"] == "attention" else None
        got.append((r, total - r if total is not None else int(tokens * part)))
    return got


def _pages(tokens):
    return -(-tokens // PAGE)


def work(c):
    if c["op"] == "logprobs":
        return {"bytes": c["rows"] * (2 * c["vocab"] + 12 + 8 * c["top"]), "flops": c["rows"] * c["vocab"] * 6}
    lens = _lengths(c)
    hk, d = c["kv_heads"], c["dim"]
    token = hk * d * 9 // 8                       # keys and values of a token in the cache: 4.5 bits each
    rows = sum(r for r, _ in lens) + c.get("pad", 0)
    if c["op"] == "read":
        return {"bytes": rows * (4 * hk * d + 4) + (rows - c["pad"]) * token, "flops": 4 * rows * hk * d}
    hq = c["q_heads"]
    if c["op"] == "append":                       # read: queries, keys, values; written: queries, the cache, and
        here = rows - c["pad"]                    # the values that it holds
        return {"bytes": rows * ((2 * hq + 2 * hk) * d * 2 + 8) + here * token + rows * 4 * hk * d,
                "flops": rows * (hq + hk) * d * 8 + 8 * rows * hk * d}
    read = pairs = 0
    w = c["window"]
    for r, p in lens:
        if not r:
            continue
        read += p + r - (max(0, p + 1 - w) if w else 0)
        for i in range(r):
            pairs += min(p + i + 1, w) if w else p + i + 1
    return {"bytes": read * token + rows * hq * d * 4, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(pages, heads, dim, gen):
    """A cache of normal values, some dimensions larger than others, as an append would leave it."""
    def one(groups, lanes):
        x = torch.randn(groups + (16,), device=DEV, generator=gen)
        x *= torch.exp(0.5 * torch.randn((1, heads) + groups[2:] + (1,), device=DEV, generator=gen))
        scale = (x.abs().amax(-1) / (6 * UNIT)).to(torch.float8_e4m3fn)
        x /= (scale.float() * UNIT).clamp(min=1e-9)[..., None]
        middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        codes = torch.bucketize(x.abs(), middle, out_int32=True).to(torch.uint8) | (x < 0).to(torch.uint8) * 8
        codes = codes.view(pages, heads, dim // 32, 64, 16, 2)
        return (codes[..., 0] | codes[..., 1] << 4).contiguous(), scale.view(lanes)
    # groups in the order in which the scales lie; the codes of one lie elsewhere for values, whose
    # groups are drawn alike
    k, ks = one((pages, heads, dim // 16, 64), (pages, heads, 64, dim // 16))
    v, vs = one((pages, heads, dim // 16, 64), (pages, heads, dim // 64, 16, 16))
    unit = torch.full((heads,), UNIT, device=DEV)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "k_unit": unit, "v_unit": unit.clone()}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c = case
    s = {"case": c}
    if c["op"] == "logprobs":
        rows, n = c["rows"], c["vocab"]
        z = 2.5 * torch.randn(rows, n, device=DEV, generator=gen)
        # a few tokens that the model is rather sure of
        sure = torch.randint(0, n, (rows, 4), device=DEV, generator=gen)
        z.scatter_add_(1, sure, 12 * torch.rand(rows, 4, device=DEV, generator=gen))
        s["logits"] = z.half()
        z = s["logits"].float() / c["temperature"]
        z -= torch.log(-torch.log(torch.rand(rows, n, device=DEV, generator=gen).clamp_(1e-30, 1 - 1e-7)))
        s["tokens"] = z.argmax(dim=1).to(torch.int32)
        f32, i32 = torch.float32, torch.int32
        s["out"] = (torch.empty(rows, dtype=f32, device=DEV), torch.empty(rows, dtype=f32, device=DEV),
                    torch.empty(rows, c["top"], dtype=i32, device=DEV),
                    torch.empty(rows, c["top"], dtype=f32, device=DEV))
        return s
    lens = s["lens"] = _lengths(c)
    hk, d = c["kv_heads"], c["dim"]
    starts = [0]
    for r, _ in lens:
        starts.append(starts[-1] + r)
    if c["op"] == "attention":
        hq = c["q_heads"]
        need = [_pages(p + r) for r, p in lens]
        s["cache"] = _cache(sum(need) + 1, hk, d, gen)
        ids = torch.randperm(sum(need) + 1, device=DEV, generator=gen).to(torch.int32)
        s["table"] = torch.zeros(len(lens), max(need) + 1, dtype=torch.int32, device=DEV)
        grid = torch.arange(max(need) + 1, device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
        s["table"][grid] = ids[:sum(need)]
        s["row_start"], s["seq_lens"] = _ints(starts), _ints([p + r for r, p in lens])
        # queries of twice unit size: scores spread by two and more
        s["q"] = (2 * torch.randn(max(1, starts[-1]), hq * d, device=DEV, generator=gen)).half()
        s["out"] = torch.zeros_like(s["q"])
        s["max_rows"] = max(r for r, _ in lens)
    else:
        pages = sum(_pages(p + r) - p // PAGE if r else 0 for r, p in lens) + 2
        s["cache"] = _cache(pages, hk, d, gen)
        ids = torch.randperm(pages, device=DEV, generator=gen)
        slots, positions, page = [], [], 0
        for r, p in lens:
            at = torch.arange(p, p + r, device=DEV)
            slots.append(ids[page + at // PAGE - p // PAGE] * PAGE + at % PAGE)
            positions.append(at)
            page += _pages(p + r) - p // PAGE if r else 0
        none = torch.zeros(c["pad"], dtype=torch.long, device=DEV)
        s["slots"] = torch.cat(slots + [none - 1]).to(torch.int32)
        rows = starts[-1] + c["pad"]
        half = lambda *shape: torch.empty(*shape, dtype=torch.float16, device=DEV)  # noqa: E731
        s["k_out"], s["v_out"] = half(rows, hk * d), half(rows, hk * d)
        if c["op"] == "append":
            hq = c["q_heads"]
            s["positions"] = torch.cat(positions + [none]).to(torch.int32)
            s["qkv"] = (torch.randn(rows, (hq + 2 * hk) * d, device=DEV, generator=gen)
                        * torch.exp(0.3 * torch.randn(rows, 1, device=DEV, generator=gen))).half()
            near = lambda: (1 + 0.2 * torch.randn(d, device=DEV, generator=gen)).half()  # noqa: E731
            s["q_weight"], s["k_weight"] = (near(), near()) if c["norm"] else (None, None)
            pairs = c["rot"] // 2
            s["inv_freq"] = (1e6 ** (-torch.arange(pairs, device=DEV, dtype=torch.float64) / pairs)).float()
            s["out"] = half(rows, hq * d)
    if own:
        from fp8_quantized_skinny_qpn_amd import kv
        s["handle"] = kv.KvCache4(**s["cache"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention,
            "logprobs": _plain_logprobs}[op](s)


def _run_own(s, op):
    from fp8_quantized_skinny_qpn_amd import kv
    c = s["case"]
    if op == "append":
        q = kv.rope_append(s["handle"], s["qkv"], c["q_heads"], s["positions"], s["slots"],
                           s["inv_freq"], s["q_weight"], s["k_weight"], EPS, c["interleaved"],
                           out=s["out"])
        k, v = kv.read(s["handle"], s["slots"], out=(s["k_out"], s["v_out"]))
        return {"q": q, "k": k, "v": v}
    if op == "read":
        k, v = kv.read(s["handle"], s["slots"], out=(s["k_out"], s["v_out"]))
        return {"k": k, "v": v}
    if op == "attention":
        return kv.attention(s["handle"], s["q"], s["row_start"], s["seq_lens"], s["table"],
                            s["max_rows"], c["dim"] ** -0.5, c["window"], out=s["out"])
    logprob, entropy, ids, alternatives = kv.logprobs(s["logits"], s["tokens"], c["top"], c["temperature"],
                                                      out=s["out"])
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids, "top_logprobs": alternatives}


# ---------------------------------------------------------------- plain forms

def _e2m1():
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.cat([v, -v])


def _pairs():
    """The two values of each byte."""
    v, b = _e2m1(), torch.arange(256, device=DEV)
    return torch.stack([v[b & 15], v[b >> 4]], -1)


def _plain_keys(b, blocks):
    """Keys of the blocks [n] (page * heads + head): [n, 64, D] in 32 bits."""
    pages, heads, rows = b["k"].shape[:3]
    g = rows // 2
    x = _pairs()[b["k"].view(pages * heads, -1)[blocks].int()]
    scale = b["k_scale"].view(pages * heads, 4, 16, 4, g)[blocks].float()         # [n, g, c, t, i]
    x = x.view(-1, rows, 4, 16, 2, 16).permute(0, 1, 4, 2, 3, 5)                  # [n, row, half, g, c, e]
    x = x.reshape(-1, 4, g, 4, 16, 16).permute(0, 1, 4, 3, 2, 5)                  # [n, t, c, g, i, e]
    x = x * scale.permute(0, 3, 2, 1, 4)[..., None]
    return x.reshape(-1, PAGE, 64 * g) * b["k_unit"][blocks % heads][:, None, None]


def _plain_values(b, blocks):
    pages, heads, rows = b["v"].shape[:3]
    g = rows // 2
    x = _pairs()[b["v"].view(pages * heads, -1)[blocks].int()]
    scale = b["v_scale"].view(pages * heads, g, 4, 4, 4, 4)[blocks].float()       # [n, i, g, a, t, r]
    x = x.view(-1, rows, 4, 4, 4, 32).permute(0, 2, 3, 4, 1, 5)                   # [n, g, a, b, row, byte]
    x = x.reshape(-1, 4, 4, 4, 4, 4, g, 4).permute(0, 4, 1, 5, 2, 6, 7, 3)        # [n, t, g, r, a, i, j, b]
    x = x * scale.permute(0, 4, 2, 5, 3, 1)[..., None, None]
    return x.reshape(-1, PAGE, 64 * g) * b["v_unit"][blocks % heads][:, None, None]


def _plain_rows(values, b, slots):
    """Rows [rows, heads * D] of the slots; zeros where there is none."""
    pages, heads = b["k"].shape[:2]
    keep = (slots >= 0) & (slots < pages * PAGE)
    at = torch.where(keep, slots, 0)
    x = values(b, torch.arange(pages * heads, device=DEV)).view(pages, heads, PAGE, -1)[at // PAGE, :, at % PAGE]
    return torch.where(keep[:, None], x.reshape(len(slots), -1), 0.0)


def _plain_read(s):
    b, slots = s["cache"], s["slots"].long()
    return {"k": _plain_rows(_plain_keys, b, slots).half(), "v": _plain_rows(_plain_values, b, slots).half()}


def _rotated(x, weight, s):
    """Norm and rotation of [rows, heads, dim] in x's type; angles in 64 bits."""
    c = s["case"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
    angle = (s["positions"].double()[:, None] * s["inv_freq"].double()[None, :])[:, None, :]
    cos, sin = torch.cos(angle).to(x.dtype), torch.sin(angle).to(x.dtype)
    turned, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :c["rot"] // 2], turned[..., c["rot"] // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, rest], -1)


def _even(x, least, bits):
    """x (64 bits, not negative) to the nearest number with `bits` bits behind the point of its binade
    (2 ** least the lowest), ties to the even one."""
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp(min=least).double() - bits)
    return torch.round(x / step) * step


def _quantised(x, unit):
    """Codes [rows, heads, groups, 16] and scales [rows, heads, groups] of x [rows, heads, D] in 64 bits."""
    x = x.unflatten(-1, (-1, 16))
    unit = unit.double()[:, None]
    scale = _even((x.abs().amax(-1) / (6 * unit)).clamp(max=448.0), -6, 3).clamp(max=448.0)
    by = torch.where(scale > 0, scale * unit, math.inf)
    size = _even((x.abs() / by[..., None]).clamp(max=6.0), 0, 1)
    code = torch.bucketize(size.float() - 0.125, _e2m1()[:8])
    code = code + torch.where((x < 0) & (scale > 0)[..., None], 8, 0)
    return code.to(torch.uint8), scale.float().to(torch.float8_e4m3fn)


def _plain_append(s):
    c, b = s["case"], s["cache"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    rows, g = s["qkv"].shape[0], d // 64
    x = s["qkv"].view(rows, hq + 2 * hk, d)
    q = _rotated(x[:, :hq].float(), s["q_weight"], s)
    # keys next to a border between two codes need their 64 bits
    k = _rotated(x[:, hq:hq + hk].double(), s["k_weight"], s)
    slots = s["slots"].long()
    at = torch.nonzero(slots >= 0).flatten()                 # (the slots of a call are all different)
    page, token = slots[at] // PAGE, slots[at] % PAGE
    t, c16 = token // 16, token % 16
    g4, r4 = token // 4 % 4, token % 4
    # keys: dimension (g, i, e) is code e of the group (t, i) of lane (g, c)
    code, scale = _quantised(k[at], b["k_unit"])
    code = (code[..., 0::2] | code[..., 1::2] << 4).view(-1, hk, 4, g, 8)
    i = torch.arange(g, device=DEV)
    n = t[:, None] * g + i                                    # [row, i]
    keys = b["k"].view(-1, hk, 2 * g, 4, 16, 2, 8)            # [page, head, row, g, c, half, byte]
    keys[page[:, None], :, n // 2, :, c16[:, None], n % 2] = code.permute(0, 3, 1, 2, 4)
    scales = b["k_scale"].view(torch.uint8).view(-1, hk, 4, 16, 4, g)
    scales[page, :, :, c16, t] = scale.view(torch.uint8).view(-1, hk, 4, g)
    # values: dimension (a, i, j, b) is code (i, j) of the token (t, r) of lane (g, a, b)
    code, scale = _quantised(x[:, hq + hk:][at].double(), b["v_unit"])
    code = code.view(-1, hk, 4, g, 2, 2, 4)                   # [row, head, a, i, j / 2, j % 2, b]
    code = (code[..., 0, :] | code[..., 1, :] << 4).permute(0, 1, 2, 5, 3, 4)
    code = code.reshape(-1, hk, 4, 4, 2 * g)                  # [row, head, a, b, byte (i, j / 2)]
    byte = (4 * t + r4)[:, None] * 2 * g + torch.arange(2 * g, device=DEV)
    values = b["v"].view(-1, hk, 2 * g, 4, 4, 4, 16)          # [page, head, row, g, a, b, byte]
    values[page[:, None], :, byte // 16, g4[:, None], :, :, byte % 16] = code.permute(0, 4, 1, 2, 3)
    scales = b["v_scale"].view(torch.uint8).view(-1, hk, g, 4, 4, 16)    # [page, head, i, g, a, (t, r)]
    scales[page, :, :, g4, :, 4 * t + r4] = scale.view(torch.uint8).view(-1, hk, 4, g).transpose(2, 3)
    return {"q": q.reshape(rows, hq * d).half(), **_plain_read(s)}


def _plain_attention(s):
    c, b = s["case"], s["cache"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    table, group = s["table"].long(), hq // hk
    n, width = table.shape
    start, total = s["row_start"][:-1].long(), s["seq_lens"].long()
    rows = s["row_start"][1:].long() - start
    most, tokens = s["max_rows"], width * PAGE
    blocks = (table[:, None, :] * hk + torch.arange(hk, device=DEV)[None, :, None]).flatten()   # [n, head, page]
    k = _plain_keys(b, blocks).view(n, hk, tokens, d)
    v = _plain_values(b, blocks).view(n, hk, tokens, d)
    i = torch.arange(most, device=DEV)
    at = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(n, most, hk, group, d).permute(0, 2, 1, 3, 4).reshape(n, hk, most * group, d)
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()) * d ** -0.5
    position = total[:, None] - rows[:, None] + i
    j = torch.arange(tokens, device=DEV)
    sees = (j <= position[..., None]) & (i < rows[:, None])[..., None]
    if c["window"]:
        sees &= j > position[..., None] - c["window"]
    sees = sees[:, None, :, None, :].expand(n, hk, most, group, tokens).reshape(n, hk, most * group, tokens)
    scores = torch.where(sees, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), 0.0, top))
    weight = p.sum(-1, keepdim=True)
    y = torch.matmul(p, v) / torch.where(weight > 0, weight, 1.0)
    y = y.view(n, hk, most, group, d).permute(0, 2, 1, 3, 4).reshape(n, most, hq * d)
    t = torch.arange(s["q"].shape[0], device=DEV)
    r = torch.searchsorted(s["row_start"][1:].long().contiguous(), t, right=True).clamp(max=n - 1)
    y = y[r, (t - start[r]).clamp(0, most - 1)]
    return torch.where((t < s["row_start"][-1])[:, None], y, 0.0).half()


def _plain_logprobs(s):
    c = s["case"]
    z = s["logits"].float()
    x = (z - z.amax(1, keepdim=True)) / c["temperature"]
    e = torch.exp(x)
    total = e.sum(1)
    log_total = torch.log(total)
    logprob = x.gather(1, s["tokens"].long()[:, None])[:, 0] - log_total
    entropy = log_total - (e * x).sum(1) / total
    _, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)   # ties: the lowest index first
    ids = ids[:, :c["top"]].contiguous()
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids.to(torch.int32),
            "top_logprobs": x.gather(1, ids) - log_total[:, None]}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attention": _exact_attention,
            "logprobs": _exact_logprobs}[case["op"]](s)


def _value_of_code(code):
    """E2M1: a sign, two bits of exponent, one of fraction."""
    exponent, fraction = (code >> 1) & 3, (code & 1).double()
    size = torch.where(exponent == 0, 0.5 * fraction, (1 + 0.5 * fraction) * 2.0 ** (exponent.double() - 1))
    return torch.where(code >= 8, -size, size)


def _code_at(block, place):
    """Half byte `place` of a block's bytes [..., bytes]."""
    byte = block[..., place // 2].int()
    return torch.where(place % 2 == 1, byte >> 4, byte & 15)


def _exact_tokens(b, pages, kind):
    """[heads, pages * 64, D] of the listed pages in 64 bits: every element looked up by itself."""
    heads, d = b["k"].shape[1], 32 * b["k"].shape[2]
    g = d // 64
    token = torch.arange(PAGE, device=DEV)[:, None]
    dim = torch.arange(d, device=DEV)[None, :]
    if kind == "k":
        t, c = token // 16, token % 16
        lane, n = dim // (16 * g) * 16 + c, t * g + dim // 16 % g
        byte = (n // 2) * 1024 + lane * 16 + (n % 2) * 8 + dim % 16 // 2
        place, at = 2 * byte + dim % 2, lane * 4 * g + n
    else:
        t, g4, r = token // 16, token // 4 % 4, token % 4
        a, i, j, low = dim // (16 * g), dim // 16 % g, dim // 4 % 4, dim % 4
        lane, half = 16 * g4 + 4 * a + low, (4 * t + r) * 4 * g + 4 * i + j
        place = 2 * ((half // 32) * 1024 + lane * 16) + half % 32
        at = (i * 16 + 4 * g4 + a) * 16 + 4 * t + r
    code = _code_at(b[kind][pages].flatten(2), place.flatten())
    scale = b[kind + "_scale"][pages].flatten(2).double()[..., at.expand(PAGE, d).flatten()]
    x = _value_of_code(code) * scale * b[kind + "_unit"].double()[None, :, None]
    return x.view(len(pages), heads, PAGE, d).transpose(0, 1).reshape(heads, -1, d)


def _exact_read(s):
    out = {}
    for kind in ("k", "v"):
        rows = torch.zeros(s[kind + "_out"].shape, dtype=torch.float64, device=DEV)
        slots = s["slots"].long()
        for page in range(0, s["cache"]["k"].shape[0], 64):
            some = torch.arange(page, min(page + 64, s["cache"]["k"].shape[0]), device=DEV)
            x = _exact_tokens(s["cache"], some, kind)
            here = torch.nonzero((slots >= page * PAGE) & (slots < (page + len(some)) * PAGE)).flatten()
            rows[here] = x[:, slots[here] - page * PAGE].transpose(0, 1).flatten(1)
        out[kind] = rows
    return out


def _nearest(x, table):
    """The index of the entry of an ascending table that is nearest to each x >= 0, the even one of two."""
    middle = (table[1:] + table[:-1]) / 2
    low = torch.searchsorted(middle, x.contiguous())         # at a tie the lower of the two
    last = len(middle) - 1
    return low + ((low <= last) & (x == middle[low.clamp(max=last)]) & (low % 2 == 1)).long()


def _exact_append(s):
    c, b = s["case"], s["cache"]
    hq, hk, d, half = c["q_heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    x = s["qkv"].double().view(-1, hq + 2 * hk, d)
    scales = [(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    scales = torch.tensor(scales[:127], dtype=torch.float64, device=DEV)
    codes = _value_of_code(torch.arange(8, device=DEV))
    got = {"q": [], "k": [], "v": []}
    turn = torch.outer(s["positions"].double(), s["inv_freq"].double())
    j = torch.arange(half, device=DEV)
    ia, ib = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
    for h in range(hq + 2 * hk):
        u = x[:, h].clone()
        if h < hq + hk:
            w = s["q_weight"] if h < hq else s["k_weight"]
            if w is not None:
                u = u / torch.sqrt(u.pow(2).sum(1) / d + EPS)[:, None] * w.double()
            p, q = u[:, ia], u[:, ib]
            u[:, ia], u[:, ib] = p * turn.cos() - q * turn.sin(), q * turn.cos() + p * turn.sin()
        if h < hq:
            got["q"].append(u)
            continue
        kind, head = ("k", h - hq) if h < hq + hk else ("v", h - hq - hk)
        unit = float(b[kind + "_unit"][head])
        for lo in range(0, d, 16):
            part = u[:, lo:lo + 16]
            scale = scales[_nearest(part.abs().amax(1) / (6 * unit), scales)][:, None]
            size = codes[_nearest(part.abs() / torch.where(scale > 0, scale * unit, 1e300), codes)]
            got[kind].append(torch.copysign(size, part) * scale * unit)
    there = (s["slots"] >= 0)[:, None]
    q, k, v = (torch.cat(got[n], 1) for n in ("q", "k", "v"))
    return {"q": q, "k": torch.where(there, k, 0.0), "v": torch.where(there, v, 0.0)}


def _exact_attention(s):
    c, b = s["case"], s["cache"]
    hq, hk, d, w = c["q_heads"], c["kv_heads"], c["dim"], c["window"]
    group = hq // hk
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for n, (rows, before) in enumerate(s["lens"]):
        if not rows:
            continue
        end = before + rows
        pages = s["table"][n, :_pages(end)].long()
        p = before + torch.arange(rows, device=DEV)
        j = torch.arange(end, device=DEV)
        hide = j[None, :] > p[:, None]
        if w:
            hide |= j[None, :] <= p[:, None] - w
        parts = [pages[i:i + 128] for i in range(0, len(pages), 128)]
        keys = torch.cat([_exact_tokens(b, part, "k") for part in parts], 1)
        values = torch.cat([_exact_tokens(b, part, "v") for part in parts], 1)
        for h in range(hk):
            k, v = keys[h, :end], values[h, :end]
            for g in range(group):
                col = (h * group + g) * d
                q = s["q"][at:at + rows, col:col + d].double()
                score = (q @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                y[at:at + rows, col:col + d] = torch.softmax(score, 1) @ v
        at += rows
    return y


def _exact_logprobs(s):
    c = s["case"]
    logprob, entropy, top = [], [], []
    for row in range(c["rows"]):
        lp = torch.log_softmax(s["logits"][row].double() / c["temperature"], 0)
        logprob.append(lp[s["tokens"][row].long()])
        entropy.append(-(lp.exp() * lp).sum())
        top.append(torch.topk(lp, c["top"])[0])
    return {"logprob": torch.stack(logprob), "entropy": torch.stack(entropy), "top_ids": None,
            "top_logprobs": torch.stack(top)}
