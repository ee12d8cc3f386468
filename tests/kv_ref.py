"""Plain FP64 references of the speculative-round operators (test infrastructure).

Written from the definitions in include/qpn_kv.h with numpy; they share no code with the kernels
or the binding.  Caches are kept as [pages, heads, 64 tokens, dim] values and scales; `pack` and
`unpack` translate to the layout the header documents.
"""
import numpy as np

PAGE = 64


def e4m3_values():
    """The value of each of the 256 codes (NaN for 0x7F and 0xFF)."""
    out = np.empty(256)
    for code in range(256):
        s, e, m = code >> 7, (code >> 3) & 15, code & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[code] = np.nan if code & 0x7F == 0x7F else (-v if s else v)
    return out


VALUES = e4m3_values()


def e4m3_codes(x):
    """Nearest E4M3 code, ties to the even code, saturating, NaN to NaN (by search over midpoints)."""
    x = np.asarray(x, np.float64)
    pos = VALUES[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    a = np.minimum(np.abs(x), 448.0)
    i = np.searchsorted(mid, a)                       # at a tie the lower code
    tie = (i < 126) & (a == mid[np.minimum(i, 125)]) & (i % 2 == 1)
    codes = (i + tie).astype(np.int64) | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), np.where(np.signbit(x), 0xFF, 0x7F), codes).astype(np.uint8)


def pack_k(codes):
    """[pages, heads, 64, dim] codes to [pages, heads, dim / 16, 64, 16]."""
    p, h, t, d = codes.shape
    return np.ascontiguousarray(codes.reshape(p, h, t, d // 16, 16).transpose(0, 1, 3, 2, 4))


def unpack_k(k):
    p, h, c, t, e = k.shape
    return np.ascontiguousarray(k.transpose(0, 1, 3, 2, 4)).reshape(p, h, t, c * e)


def pack_v(codes):
    """[pages, heads, 64, dim] codes to [pages, heads, dim, 64] (token 16 t + 4 g + r at 16 g + 4 t + r)."""
    out = np.empty(codes.shape[:2] + (codes.shape[3], PAGE), codes.dtype)
    for tok in range(PAGE):
        out[..., (tok // 4 % 4) * 16 + tok // 16 * 4 + tok % 4] = codes[:, :, tok, :]
    return out


def unpack_v(v):
    out = np.empty(v.shape[:2] + (PAGE, v.shape[2]), v.dtype)
    for tok in range(PAGE):
        out[:, :, tok, :] = v[..., (tok // 4 % 4) * 16 + tok // 16 * 4 + tok % 4]
    return out


def plan_round(before, rows, held, table, free_pages, free_count, capacity):
    """The tables, one request after another."""
    width = table.shape[1]
    table = table.copy()
    free = min(max(free_count, 0), len(free_pages))
    asked_pages = asked_rows = taken = at = 0
    seq, start, held_out, slots, positions = [], [0], [], [], []
    for r, (b, n, h) in enumerate(zip(before, rows, held)):
        need = -(-(b + n) // PAGE)
        fine = b >= 0 and n >= 0 and 0 <= h <= width and need <= width and b <= h * PAGE
        want = max(0, need - h) if fine else 0
        go = False
        if fine:
            asked_pages += want
            asked_rows += n
            go = asked_pages <= free and asked_rows <= capacity
        if go:
            for j in range(want):
                table[r, h + j] = free_pages[free - 1 - taken]
                taken += 1
            for i in range(n):
                p = b + i
                slots.append(int(table[r, p // PAGE]) * PAGE + p % PAGE)
                positions.append(p)
            at += n
        seq.append(b + (n if go else 0) if fine else 0)
        held_out.append(h + (want if go else 0))
        start.append(at)
    pad = capacity - len(slots)
    return dict(seq_lens=seq, row_start=start, held=held_out, free_count=[free - taken], table=table,
                slots=slots + [-1] * pad, positions=positions + [0] * pad)


def norm_rope(x, weight, eps, inv_freq, interleaved, positions):
    """x [rows, heads, dim] normed per head and rotated, in 64 bits."""
    x = np.asarray(x, np.float64).copy()
    d = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / d + eps) * np.asarray(weight, np.float64)
    half = len(inv_freq)
    ang = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang), np.sin(ang)
    j = np.arange(half)
    ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def page_scale(amax):
    s = 2.0 ** -60
    while 448 * s < amax:
        s *= 2
    return s


def append(codes, scale, x, slots):
    """x [rows, heads, dim] into codes [pages, heads, 64, dim] and scale [pages, heads] (in place)."""
    rows_of = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < codes.shape[0] * PAGE:
            rows_of.setdefault(slot // PAGE, {})[slot % PAGE] = t   # the later row of one slot counts
    for page, places in rows_of.items():
        offs = sorted(places)
        rest = [o for o in range(PAGE) if o not in places]
        for h in range(codes.shape[1]):
            new = np.stack([x[places[o], h] for o in offs])
            fin = np.abs(new[np.isfinite(new)])
            s = page_scale(fin.max() if fin.size else 0.0)
            old = 0.0 if 0 in places else float(scale[page, h])
            now = max(s, old)
            if old > 0 and now > old:
                codes[page, h, rest] = e4m3_codes(VALUES[codes[page, h, rest]] * (old / now))
            codes[page, h, offs] = e4m3_codes(new / now)
            scale[page, h] = now


def attention(q, k, v, row_start, seq_lens, table, scale, window):
    """y and, per output, the mean |v| under the weights and the weights' sum against the row's
    maximum (for tolerances).  k, v: [pages, heads, 64, dim] values; q [rows, q_heads, dim]."""
    rows, hq, d = q.shape
    hk = k.shape[1]
    y, mag = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    for r in range(len(seq_lens)):
        n = row_start[r + 1] - row_start[r]
        pages = -(-max(seq_lens[r], 0) // PAGE)
        ids = table[r, :pages]
        for h in range(hq):
            kk = k[ids, h * hk // hq].reshape(-1, d)
            vv = v[ids, h * hk // hq].reshape(-1, d)
            for i in range(n):
                p = seq_lens[r] - n + i
                lo = max(0, p - window + 1) if window else 0
                if p < lo:
                    continue
                s = scale * (kk[lo:p + 1] @ q[row_start[r] + i, h])
                w = np.exp(s - s.max())
                y[row_start[r] + i, h] = w @ vv[lo:p + 1] / w.sum()
                mag[row_start[r] + i, h] = w @ np.abs(vv[lo:p + 1]) / w.sum()
    return y, mag


def softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def verify(logits, draft_logits, tokens, row_start, inv_temperature, accept_u, sample_u):
    n = logits.shape[1]
    accepted, nxt, prob = [], [], np.zeros(len(logits))
    for r in range(len(row_start) - 1):
        a, b = row_start[r], row_start[r + 1]
        if b <= a:
            accepted.append(0)
            nxt.append(-1)
            continue
        stop = None
        for t in range(a, b - 1):
            d = tokens[t + 1]
            p = softmax(logits[t].astype(np.float64) * inv_temperature)
            q = softmax(draft_logits[t].astype(np.float64) * inv_temperature) if draft_logits is not None else None
            pd, qd = (p[d], 1.0 if q is None else q[d]) if 0 <= d < n else (0.0, 0.0)
            prob[t] = 0.0 if not 0 <= d < n else 1.0 if pd >= qd else pd / qd
            if stop is None and not (0 <= d < n and accept_u[t] * qd < pd):
                stop = t
        if stop is None:
            w = softmax(logits[b - 1].astype(np.float64) * inv_temperature)
            accepted.append(b - 1 - a)
        else:
            p = softmax(logits[stop].astype(np.float64) * inv_temperature)
            if draft_logits is None:
                w = p.copy()
                if 0 <= tokens[stop + 1] < n:
                    w[tokens[stop + 1]] = 0
            else:
                w = np.maximum(p - softmax(draft_logits[stop].astype(np.float64) * inv_temperature), 0)
            if not w.sum() > 0:
                w = p
            accepted.append(stop - a)
        up = np.cumsum(w)
        x = int((up <= float(sample_u[r]) * up[-1]).sum())
        some = np.nonzero(w > 0)[0]
        nxt.append(min(x, int(some[-1])) if some.size else -1)
    return accepted, nxt, prob
