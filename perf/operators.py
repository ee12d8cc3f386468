"""The operators of a speculative round over an 8-bit paged KV cache: what is measured.

Four operators stand around the packed-weight products of a decoder layer:

  plan        block tables, slot map and positions of a round from the requests' lengths
  append      norms of queries and keys per head with the position rotation, keys and values
              written to the cache as E4M3 codes with a power-of-two scale per page and head
  attention   attention of a round's rows over that cache
  verify      drafted tokens against the target's probabilities, from given random numbers

The cache holds pages of 64 tokens.  Per page and KV head of D dimensions:
  keys    [D / 16, 64, 16]: dimension 16 c + e of token t at [c, t, e];
  values  [D, 4, 4, 4]: dimension d of token 16 t + 4 g + r at [d, g, t, r];
  one float32 scale each: a value is its code times the scale.

Sizes: 40 query and 8 key/value heads of 128 dimensions make the 7168 output channels of the
QKV projection that the benchmark times (10 and 2 heads on one of four tensor-parallel shards),
8 rows are its verify block, 256 rows its largest prefill block, 151936 its vocabulary.
"""
import math

import torch

own = False

PAGE = 64
SCALE_FLOOR = 2.0 ** -60   # the scale of a page that holds nothing but zeros
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


def _verify(name, requests, rows, vocab, sampled, temperature):
    return dict(name=name, op="verify", requests=requests, rows=rows, vocab=vocab,
                sampled=sampled, temperature=temperature)


def _plan(name, requests, rows, tokens, short=False):
    return dict(name=name, op="plan", requests=requests, rows=rows, tokens=tokens, short=short)


def listed():
    return [
        # one request's verify round begins: 8 rows after 4090 tokens
        _plan("plan 1 request", 1, 8, 4090),
        # a server's round: 256 requests of up to 8 rows, tables of up to 513 pages
        _plan("plan 256 requests", 256, 8, 32768),
        # plain decoding, one token of one request
        _append("append 1 row", 1, 1, 1777),
        # the verify block: the last token and seven drafts, across a page's end
        _append("append 8 rows", 1, 8, 4090),
        # prompt blocks of four requests
        _append("append 4x256 rows", 4, 256, 1000),
        # the first tokens of an answer: latency alone
        _attn("attention 1 row 200", 1, 1, 200),
        # the verify block over a chat's history
        _attn("attention 8 rows 4099", 1, 8, 4099),
        # the verify block over a long document: the cache's bytes are all that counts
        _attn("attention 8 rows 131k", 1, 8, 131001),
        # many requests on one of four tensor-parallel shards, lengths and rows ragged
        _attn("attention 48 ragged", 48, 8, 9000, 10, 2, 128, 0, True),
        # a prompt block of 256 rows late in a long prompt: matrix work
        _attn("attention 256 rows 20k", 1, 256, 20001),
        # the round's end: seven drafts of a greedy drafter over the full vocabulary
        _verify("verify 8 rows greedy", 1, 8, 151936, False, 0.8),
        # 32 requests with sampled drafts
        _verify("verify 32x8 sampled", 32, 8, 151936, True, 1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "append", "append", "attention", "attention", "attention", "verify"])
    if kind == "plan":
        c = _plan("", _log_int(rng, 1, 256), rng.randint(1, 8), _log_int(rng, 10, 32768),
                  rng.random() < 0.4)
    elif kind == "append":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        dim = rng.choice([64, 128, 128, 256])
        while kv_heads * group * dim > 5120:
            group = max(1, group // 2)
            kv_heads = max(1, kv_heads // 2) if group == 1 else kv_heads
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        requests = _log_int(rng, 1, 32)
        rows = min(_log_int(rng, 1, 256), max(1, 1024 // requests))
        c = _append("", requests, rows, _log_int(rng, 1, 200000), kv_heads * group, kv_heads, dim,
                    rot, rng.random() < 0.3, rng.random() < 0.8, rng.choice([0, 0, 3]))
    elif kind == "attention":
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        dim = rng.choice([64, 128, 128, 256])
        while kv_heads * group * dim > 5120:
            group = max(1, group // 2)
            kv_heads = max(1, kv_heads // 2) if group == 1 else kv_heads
        requests = _log_int(rng, 1, 64)
        rows = rng.choice([1, 1, 4, 8, 8, rng.randint(2, 8), _log_int(rng, 9, 256)])
        room = 128000 * 8 * 128 // (requests * kv_heads * dim)
        room = min(room, 200_000_000 // (requests * kv_heads * group * rows))
        tokens = _log_int(rng, 30, max(31, min(131000, room)))
        if rows > 8:
            tokens = max(rows, min(tokens, 20000 * 256 * 5120 // (rows * requests * kv_heads * group * dim)))
        window = rng.choice([0, 0, 0, rng.randint(1, max(2, tokens))])
        c = _attn("", requests, rows, tokens, kv_heads * group, kv_heads, dim, window,
                  requests > 1)
    else:
        c = _verify("", _log_int(rng, 1, 31), rng.randint(1, 8), _log_int(rng, 1000, 151936),
                    rng.random() < 0.5, rng.choice([0.3, 0.7, 1.0, 1.3]))
    del c["name"]
    return c


# ---------------------------------------------------------------- lengths (of the case alone)

def _lengths(c):
    """(rows, tokens before them) of each request."""
    n, rows, tokens = c["requests"], c["rows"], c.get("tokens", 0)
    got = []
    for i in range(n):
        part = 1.0 if i == 0 else (i * 0.6180339887498949) % 1.0
        r = rows if i == 0 or not c.get("ragged", c["op"] == "plan") else (i * 5 + 3) % (rows + 1)
        total = max(r, int(tokens * part), 1) if c["op"] == "attention" else None
        got.append((r, total - r if total is not None else int(tokens * part)))
    return got


def _pages(tokens):
    return -(-tokens // PAGE)


def work(c):
    lens = _lengths(c)
    if c["op"] == "plan":
        new = sum(max(0, _pages(p + r) - _pages(p)) for r, p in lens)
        return {"bytes": 28 * len(lens) + 8 * sum(r for r, _ in lens) + 8 * new, "flops": 0}
    if c["op"] == "append":
        rows = sum(r for r, _ in lens) + c["pad"]
        hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
        return {"bytes": rows * ((2 * hq + 2 * hk) * d * 2 + 8) + (rows - c["pad"]) * 2 * hk * d,
                "flops": rows * (hq + hk) * d * 8}
    if c["op"] == "attention":
        hq, hk, d, w = c["q_heads"], c["kv_heads"], c["dim"], c["window"]
        read = pairs = 0
        for r, p in lens:
            if not r:
                continue
            first = max(0, p + 1 - w) if w else 0
            read += p + r - first
            for i in range(r):
                pairs += min(p + i + 1, w) if w else p + i + 1
        rows = sum(r for r, _ in lens)
        return {"bytes": read * hk * 2 * d + _pages(read) * 8 * hk + rows * hq * d * 4,
                "flops": 4 * d * hq * pairs}
    rows = sum(r for r, _ in lens)
    return {"bytes": rows * c["vocab"] * (4 if c["sampled"] else 2) + rows * 12 + 12 * len(lens),
            "flops": rows * c["vocab"] * (20 if c["sampled"] else 10)}


# ---------------------------------------------------------------- inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cache(pages, heads, dim, gen):
    """Codes of normal values with a scale for each page and head."""
    def one(shape):
        x = torch.randn((pages, heads) + shape, device=DEV, generator=gen)
        size = torch.exp(0.4 * torch.randn((pages, heads), device=DEV, generator=gen))
        top = x.abs().amax(dim=tuple(range(2, x.dim())))
        codes = (x * (440.0 / top).view(pages, heads, *([1] * len(shape)))).to(torch.float8_e4m3fn)
        return codes, torch.exp2(torch.ceil(torch.log2(size * top / 448.0)))
    k, ks = one((dim // 16, PAGE, 16))
    v, vs = one((dim, PAGE))
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c, lens = case, _lengths(case)
    s = {"case": c, "lens": lens}
    starts = [0]
    for r, _ in lens:
        starts.append(starts[-1] + r)
    if c["op"] == "plan":
        width = _pages(max(p + r for r, p in lens) + 1) + 1
        held = [_pages(p) for _, p in lens]
        new = sum(max(0, _pages(p + r) - h) for (r, p), h in zip(lens, held))
        total = sum(held) + new + 5
        ids = torch.randperm(total, device=DEV, generator=gen).to(torch.int32)
        s["table"] = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
        grid = torch.arange(width, device=DEV)[None, :] < torch.tensor(held, device=DEV)[:, None]
        s["table"][grid] = ids[:sum(held)]
        s["free"] = ids[sum(held):].contiguous()
        s["free_count"] = _ints([(new + 1) // 2 if c["short"] else new + 5])
        s["before"], s["rows"], s["held"] = _ints([p for _, p in lens]), _ints([r for r, _ in lens]), _ints(held)
        s["capacity"] = max(1, starts[-1])
        s["out"] = {k: torch.zeros(n, dtype=torch.int32, device=DEV) for k, n in (
            ("seq_lens", len(lens)), ("row_start", len(lens) + 1), ("held", len(lens)),
            ("free_count", 1), ("slots", s["capacity"]), ("positions", s["capacity"]))}
    elif c["op"] == "append":
        hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
        touched = sum(_pages(p + r) - p // PAGE if r else 0 for r, p in lens)
        pages = touched + 2
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
        s["positions"] = torch.cat(positions + [none]).to(torch.int32)
        rows = starts[-1] + c["pad"]
        s["qkv"] = (torch.randn(rows, (hq + 2 * hk) * d, device=DEV, generator=gen)
                    * torch.exp(0.3 * torch.randn(rows, 1, device=DEV, generator=gen))).half()
        near = lambda: (1 + 0.2 * torch.randn(d, device=DEV, generator=gen)).half()  # noqa: E731
        s["q_weight"], s["k_weight"] = (near(), near()) if c["norm"] else (None, None)
        half = c["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        s["out"] = torch.empty(rows, hq * d, dtype=torch.float16, device=DEV)
    elif c["op"] == "attention":
        hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
        need = [_pages(p + r) for r, p in lens]
        s["cache"] = _cache(sum(need) + 1, hk, d, gen)
        ids = torch.randperm(sum(need) + 1, device=DEV, generator=gen).to(torch.int32)
        s["table"] = torch.zeros(len(lens), max(need) + 1, dtype=torch.int32, device=DEV)
        grid = torch.arange(max(need) + 1, device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
        s["table"][grid] = ids[:sum(need)]
        s["row_start"], s["seq_lens"] = _ints(starts), _ints([p + r for r, p in lens])
        # queries of twice unit size: scores spread by about two
        s["q"] = (2 * torch.randn(max(1, starts[-1]), hq * d, device=DEV, generator=gen)).half()
        s["out"] = torch.zeros_like(s["q"])
        s["max_rows"] = max(r for r, _ in lens)
    else:
        rows, n = max(1, starts[-1]), c["vocab"]
        s["logits"] = (2.5 * torch.randn(rows, n, device=DEV, generator=gen)).half()
        near = (s["logits"].float() + 0.7 * torch.randn(rows, n, device=DEV, generator=gen))
        s["draft_logits"] = near.half() if c["sampled"] else None
        if c["sampled"]:  # drawn from the drafter's distribution
            near = s["draft_logits"].float() / c["temperature"]
            near -= torch.log(-torch.log(torch.rand(rows, n, device=DEV, generator=gen).clamp_(1e-30, 1 - 1e-7)))
        picked = near.argmax(dim=1).to(torch.int32)
        s["tokens"] = torch.cat([picked[:1], picked[:-1]])   # row i's drafted token is the input of row i + 1
        s["row_start"] = _ints(starts)
        s["accept_u"] = torch.rand(rows, device=DEV, generator=gen)
        s["sample_u"] = torch.rand(len(lens), device=DEV, generator=gen)
        s["out"] = (torch.empty(len(lens), dtype=torch.int32, device=DEV),
                    torch.empty(len(lens), dtype=torch.int32, device=DEV),
                    torch.empty(rows, dtype=torch.float32, device=DEV))
    if own:
        _handles(s)
    return s


def _handles(s):
    """The cache's handle and the outputs' record, which a user's program keeps."""
    from fp8_quantized_skinny_qpn_amd import kv
    if "cache" in s:
        b = s["cache"]
        s["handle"] = kv.KvCache(b["k"], b["v"], b["k_scale"], b["v_scale"])
    if s["case"]["op"] == "plan":
        s["round"] = kv.Round(**s["out"])


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention,
            "verify": _plain_verify}[op](s)


def _run_own(s, op):
    from fp8_quantized_skinny_qpn_amd import kv
    c = s["case"]
    if op == "plan":
        r = kv.plan_round(s["before"], s["rows"], s["held"], s["table"], s["free"], s["free_count"],
                          out=s["round"])
        return {"row_start": r.row_start, "seq_lens": r.seq_lens, "held": r.held,
                "free_count": r.free_count, "table": s["table"], "slots": r.slots,
                "positions": r.positions}
    if op == "append":
        q = kv.rope_append(s["handle"], s["qkv"], c["q_heads"], s["positions"], s["slots"],
                           s["inv_freq"], s["q_weight"], s["k_weight"], EPS, c["interleaved"],
                           out=s["out"])
        return {"q": q, **s["cache"]}
    if op == "attention":
        return kv.attention(s["handle"], s["q"], s["row_start"], s["seq_lens"], s["table"],
                            s["max_rows"], c["dim"] ** -0.5, c["window"], out=s["out"])
    accepted, token, prob = kv.verify_sampled(
        s["logits"], s["tokens"], s["row_start"], s["accept_u"], s["sample_u"], s["draft_logits"],
        c["temperature"], out=s["out"])
    return {"accepted": accepted, "next": token, "accept_prob": prob}


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    before, rows, held = s["before"].long(), s["rows"].long(), s["held"].long()
    table, free, count = s["table"], s["free"], s["free_count"].long()
    width, capacity = table.shape[1], s["capacity"]
    need = (before + rows + PAGE - 1) // PAGE
    fine = (before >= 0) & (rows >= 0) & (held >= 0) & (held <= width) & (need <= width) & (before <= held * PAGE)
    want = torch.where(fine, (need - held).clamp(min=0), 0)
    asked = torch.where(fine, rows, 0)
    go = fine & (torch.cumsum(want, 0) <= count) & (torch.cumsum(asked, 0) <= capacity)
    want, asked = torch.where(go, want, 0), torch.where(go, asked, 0)
    taken = torch.cumsum(want, 0) - want
    row_start = torch.cat([asked.new_zeros(1), torch.cumsum(asked, 0)])
    seq_lens = torch.where(fine, before + asked, 0)
    j = torch.arange(width, device=DEV)[None, :]
    new = (j >= held[:, None]) & (j < (held + want)[:, None])
    at = (count - 1 - taken[:, None] - (j - held[:, None])).clamp(0, free.numel() - 1)
    table.copy_(torch.where(new, free[at], table))
    t = torch.arange(capacity, device=DEV)
    r = torch.searchsorted(row_start[1:].contiguous(), t, right=True).clamp(max=rows.numel() - 1)
    used = t < row_start[-1]
    position = before[r] + t - row_start[r]
    page = table[r, (position // PAGE).clamp(0, width - 1)].long()
    slots = torch.where(used, page * PAGE + position % PAGE, -1)
    position = torch.where(used, position, 0)
    i32 = torch.int32
    return {"row_start": row_start.to(i32), "seq_lens": seq_lens.to(i32), "held": (held + want).to(i32),
            "free_count": (count - want.sum()).to(i32), "table": table, "slots": slots.to(i32),
            "positions": position.to(i32)}


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


def _e4m3(x):
    """x (64 bits) to the nearest E4M3 value, ties to the even code, saturating."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).float().to(torch.float8_e4m3fn)


def _plain_put(codes, scale, x, slots, token_at):
    """x [rows, heads, dim] in 64 bits into one cache; token_at puts codes at their tokens."""
    keep = slots >= 0
    page = torch.where(keep, slots // PAGE, 0)
    pages, heads = scale.shape
    top = torch.where(keep[:, None], x.abs().amax(-1), 0.0)
    at = page[:, None].expand(-1, heads)
    top = torch.zeros(pages, heads, dtype=x.dtype, device=DEV).scatter_reduce(0, at, top, "amax")
    first = torch.full((pages,), PAGE, device=DEV).scatter_reduce(
        0, page, torch.where(keep, slots % PAGE, PAGE), "amin")
    m, e = torch.frexp(top)
    need = torch.exp2((e - 9 + (m > 0.875)).double()).clamp(min=SCALE_FLOOR)
    need = torch.where(top > 0, need, SCALE_FLOOR)
    old = torch.where((first == 0)[:, None], 0.0, scale.double())
    new = torch.where((first < PAGE)[:, None], torch.maximum(old, need), scale.double())
    grown = (new > old) & (old > 0)
    shape = [pages, heads] + [1] * (codes.dim() - 2)
    again = _e4m3(codes.double() * (torch.where(grown, old, new) / new).view(shape))
    codes.copy_(torch.where(grown.view(shape), again.float(), codes.float()).to(torch.float8_e4m3fn))
    scale.copy_(new)
    token_at(codes, page, slots % PAGE, _e4m3(x / new[page][..., None]), keep)


def _put_keys(codes, page, offset, values, keep):
    rows, heads, dim = values.shape
    flat = codes.view(torch.uint8)
    old = flat[page, :, :, offset, :]
    values = values.view(torch.uint8).view(rows, heads, dim // 16, 16)
    at = torch.nonzero(keep).flatten()
    flat[page[at], :, :, offset[at], :] = torch.where(keep[:, None, None, None], values, old)[at]


def _put_values(codes, page, offset, values, keep):
    place = (offset // 4 % 4) * 16 + (offset // 16) * 4 + offset % 4
    at = torch.nonzero(keep).flatten()
    codes.view(torch.uint8)[page[at], :, :, place[at]] = values.view(torch.uint8)[at]


def _plain_append(s):
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    rows = s["qkv"].shape[0]
    x = s["qkv"].view(rows, hq + 2 * hk, d)
    q = _rotated(x[:, :hq].float(), s["q_weight"], s)
    # keys next to a border between two codes need their 64 bits
    k = _rotated(x[:, hq:hq + hk].double(), s["k_weight"], s)
    b, slots = s["cache"], s["slots"].long()
    _plain_put(b["k"], b["k_scale"], k, slots, _put_keys)
    _plain_put(b["v"], b["v_scale"], x[:, hq + hk:].double(), slots, _put_values)
    return {"q": q.reshape(rows, hq * d).half(), **b}


def _plain_attention(s):
    c, b = s["case"], s["cache"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    table, group = s["table"].long(), hq // hk
    n, width = table.shape
    start, total = s["row_start"][:-1].long(), s["seq_lens"].long()
    rows = s["row_start"][1:].long() - start
    most, tokens = s["max_rows"], width * PAGE
    k = b["k"][table].float() * b["k_scale"][table][..., None, None, None]   # [n, page, head, d/16, 64, 16]
    k = k.permute(0, 2, 1, 4, 3, 5).reshape(n, hk, tokens, d)
    v = b["v"][table].float() * b["v_scale"][table][..., None, None]         # [n, page, head, d, 64]
    v = v.view(n, width, hk, d, 4, 4, 4).permute(0, 2, 1, 5, 4, 6, 3).reshape(n, hk, tokens, d)
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


def _plain_verify(s):
    c = s["case"]
    inverse = 1.0 / c["temperature"]
    n, rows = c["vocab"], s["logits"].shape[0]
    start = s["row_start"].long()
    z = s["logits"].double()
    p = torch.exp((z - z.amax(1, keepdim=True)) * inverse)
    p = p / p.sum(1, keepdim=True)
    t = torch.arange(rows, device=DEV)
    drafted = s["tokens"].long()[(t + 1).clamp(max=rows - 1)]
    at = drafted[:, None]
    if s["draft_logits"] is not None:
        z = s["draft_logits"].double()
        q = torch.exp((z - z.amax(1, keepdim=True)) * inverse)
        q = q / q.sum(1, keepdim=True)
    else:
        q = torch.zeros_like(p).scatter(1, at, 1.0)
    r = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=start.numel() - 2)
    last = t >= start[r + 1] - 1          # a request's last row has no draft after it
    pd, qd = p.gather(1, at)[:, 0], q.gather(1, at)[:, 0]
    accept = (s["accept_u"].double() * qd < pd) & ~last
    prob = torch.where(last, 0.0, torch.minimum(pd / qd, torch.ones_like(pd)))
    # the first row of each request that is not accepted
    stops = torch.where(accept, rows, t)
    stop = torch.full((start.numel() - 1,), rows, device=DEV).scatter_reduce(0, r, stops, "amin")
    some = start[1:] > start[:-1]
    row = torch.where(some, stop, 0).clamp(max=rows - 1)
    rest = torch.where(last[row][:, None], p[row], (p[row] - q[row]).clamp(min=0.0))
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[row])
    up = torch.cumsum(rest, 1)
    token = (up <= s["sample_u"].double()[:, None] * up[:, -1:]).sum(1)
    highest = torch.where(rest > 0, torch.arange(n, device=DEV), -1).amax(1)
    token = torch.where(some, torch.minimum(token, highest), -1)
    accepted = torch.where(some, row - start[:-1], 0)
    return {"accepted": accepted.to(torch.int32), "next": token.to(torch.int32), "accept_prob": prob.float()}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "verify": _exact_verify}[case["op"]](s)


def _codes_table():
    """The 127 values of the E4M3 codes 0 .. 126."""
    v = [(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=DEV)


def _nearest(x):
    table = _codes_table()
    middle = (table[1:] + table[:-1]) / 2
    a = x.abs().contiguous()
    low = torch.searchsorted(middle, a)                    # at a tie the lower of the two
    tie = (low < 126) & (a == middle[low.clamp(max=125)]) & (low % 2 == 1)
    return torch.copysign(table[low + tie.long()], x)


def _exact_append(s):
    c = s["case"]
    hq, hk, d, half = c["q_heads"], c["kv_heads"], c["dim"], c["rot"] // 2
    rows = s["qkv"].shape[0]
    x = s["qkv"].double().view(rows, hq + 2 * hk, d)
    heads = []
    for h in range(hq + hk):
        u = x[:, h].clone()
        w = s["q_weight"] if h < hq else s["k_weight"]
        if w is not None:
            u = u / torch.sqrt(u.pow(2).sum(1) / d + EPS)[:, None] * w.double()
        turn = torch.outer(s["positions"].double(), s["inv_freq"].double())
        j = torch.arange(half, device=DEV)
        ia, ib = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
        a, b = u[:, ia], u[:, ib]
        u[:, ia], u[:, ib] = a * turn.cos() - b * turn.sin(), b * turn.cos() + a * turn.sin()
        heads.append(u)
    slots = s["slots"].tolist()
    by_page = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            by_page.setdefault(slot // PAGE, []).append((slot % PAGE, t))
    got = {"q": torch.cat(heads[:hq], 1)}
    for name in ("k", "v"):
        b = s["cache"]
        new = torch.stack(heads[hq:], 1) if name == "k" else x[:, hq + hk:]
        codes, scale = b[name].double(), b[name + "_scale"].double()
        for page, places in by_page.items():
            offsets = [o for o, _ in places]
            block = codes[page]                             # a view: [head, ...]
            tokens = (block.transpose(1, 2) if name == "k" else
                      block.view(hk, d, 4, 4, 4).permute(0, 3, 2, 4, 1))
            x_new = new[[t for _, t in places]].transpose(0, 1)   # [head, place, d]
            top = x_new.abs().amax((1, 2))
            for h in range(hk):
                if float(top[h]) == 0:
                    fit = SCALE_FLOOR
                else:
                    fit = 2.0 ** math.ceil(math.log2(float(top[h]) / 448.0))
                    while fit * 448.0 < float(top[h]):
                        fit *= 2
                    while fit * 224.0 >= float(top[h]):
                        fit /= 2
                fit = max(fit, SCALE_FLOOR)
                was = 0.0 if min(offsets) == 0 else float(scale[page, h])
                now = max(was, fit)
                if was and now > was:
                    block[h] = _nearest(block[h] * (was / now))
                scale[page, h] = now
            now = scale[page][:, None, None]
            put = _nearest((x_new / now).clamp(-448, 448))
            for i, o in enumerate(offsets):
                if name == "k":
                    tokens[:, o] = put[:, i].view(hk, d // 16, 16)
                else:
                    tokens[:, o // 16, o // 4 % 4, o % 4] = put[:, i]
        got[name], got[name + "_scale"] = codes, scale
    return got


def _exact_attention(s):
    c, b = s["case"], s["cache"]
    hq, hk, d, w = c["q_heads"], c["kv_heads"], c["dim"], c["window"]
    group = hq // hk
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    order = [[16 * t + 4 * g + r for t in range(4) for r in range(4)] for g in range(4)]
    order = torch.tensor([x for part in order for x in part], device=DEV)   # the token at each place
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
        for h in range(hk):
            k = b["k"][pages, h].double() * b["k_scale"][pages, h].double()[:, None, None, None]
            k = k.transpose(1, 2).reshape(-1, d)[:end]
            v = torch.empty(len(pages), PAGE, d, dtype=torch.float64, device=DEV)
            v[:, order] = (b["v"][pages, h].double() * b["v_scale"][pages, h].double()[:, None, None]).transpose(1, 2)
            v = v.reshape(-1, d)[:end]
            for g in range(group):
                col = (h * group + g) * d
                q = s["q"][at:at + rows, col:col + d].double()
                score = (q @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                y[at:at + rows, col:col + d] = torch.softmax(score, 1) @ v
        at += rows
    return y


def _exact_verify(s):
    c = s["case"]
    prob = torch.zeros(s["logits"].shape[0], dtype=torch.float64, device=DEV)
    tokens, at = s["tokens"].tolist(), 0
    for rows, _ in s["lens"]:
        for t in range(at, at + rows - 1):
            d = tokens[t + 1]
            lp = torch.log_softmax(s["logits"][t].double() / c["temperature"], 0)[d]
            lq = 0.0
            if s["draft_logits"] is not None:
                lq = torch.log_softmax(s["draft_logits"][t].double() / c["temperature"], 0)[d]
            prob[t] = torch.exp(lp - lq).clamp(max=1.0)
        at += rows
    return {"accepted": None, "next": None, "accept_prob": prob}
