"""Plain FP64 references of the 4-bit KV cache and of the log probabilities (test infrastructure).

Written from the definitions in include/qpn_kv4.h and qpn_kv.h with numpy; they share no code with
the kernels or the binding.  Caches are kept as codes [pages, heads, 64 tokens, dim] and scale codes
[pages, heads, 64 tokens, dim / 16]; `pack` and `unpack` translate to the layout the header documents.
"""
import numpy as np

import kv_ref

PAGE = 64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def places(dim):
    """For each (token, dimension): (half byte of the key codes, byte of the key scales, half byte of the
    value codes, byte of the value scales) within a block, from the header's words, one at a time."""
    g_n = dim // 64
    out = np.empty((4, PAGE, dim), np.int64)
    for tok in range(PAGE):
        for d in range(dim):
            t, c = tok // 16, tok % 16
            e, i, g = d % 16, d // 16 % g_n, d // 16 // g_n
            n, lane = t * g_n + i, 16 * g + c
            out[0, tok, d] = 2 * ((n // 2) * 64 * 16 + lane * 16 + 8 * (n % 2)) + e
            out[1, tok, d] = lane * 4 * g_n + n
            g, r = tok // 4 % 4, tok % 4
            b, j, i, a = d % 4, d // 4 % 4, d // 16 % g_n, d // 16 // g_n
            lane = 16 * g + 4 * a + b
            half = ((t * 4 + r) * g_n + i) * 4 + j            # of the lane's 64 G half bytes
            row, rest = half // 32, half % 32
            out[2, tok, d] = 2 * (row * 64 * 16 + lane * 16) + rest
            out[3, tok, d] = (i * 16 + 4 * g + a) * 16 + 4 * t + r
    return out


_PLACES = {dim: places(dim) for dim in (64, 128, 256)}


def pack(codes, scales, kind):
    """Codes and scale codes to the layout's bytes: [pages, heads, 32 dim], [pages, heads, 4 dim]."""
    p, h, _, dim = codes.shape
    at = _PLACES[dim][0 if kind == "k" else 2]
    half = np.zeros((p, h, 64 * dim), np.uint8)
    half[..., at] = codes
    sc = np.zeros((p, h, 4 * dim), np.uint8)
    sc[..., _PLACES[dim][1 if kind == "k" else 3][:, ::16]] = scales
    return half[..., 0::2] | half[..., 1::2] << 4, sc


def unpack(data, sc, dim, kind):
    data, sc = data.reshape(*data.shape[:2], 32 * dim), sc.reshape(*sc.shape[:2], 4 * dim)
    half = np.stack([data & 15, data >> 4], -1).reshape(*data.shape[:2], -1)
    return half[..., _PLACES[dim][0 if kind == "k" else 2]], sc[..., _PLACES[dim][1 if kind == "k" else 3][:, ::16]]


def values(codes, scales, unit):
    """The values that codes [..., heads, 64, dim] stand for."""
    return E2M1[codes] * np.repeat(kv_ref.VALUES[scales], 16, -1) * np.asarray(unit, np.float64)[:, None, None]


def quantise(x, unit):
    """Codes [..., dim] and scale codes [..., dim / 16] of x [..., heads, dim], by search over midpoints."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, 16)
    u = np.asarray(unit, np.float64)[:, None]
    fine = np.isfinite(g).all(-1) & (u > 0) & np.isfinite(u)
    with np.errstate(all="ignore"):
        scale = kv_ref.e4m3_codes(np.where(fine, np.abs(g).max(-1) / (6 * u), 0.0))
        step = (kv_ref.VALUES[scale] * u)[..., None]
        a = np.abs(g) / np.where(step > 0, step, 1.0)
    mid = (E2M1[1:8] + E2M1[:7]) / 2
    i = np.searchsorted(mid, np.where(np.isfinite(a), a, 0.0))          # at a tie the lower code
    tie = (i < 7) & (a == mid[np.minimum(i, 6)]) & (i % 2 == 1)
    codes = np.where(step > 0, (i + tie) | np.where(np.signbit(g), 8, 0), 0)
    codes = np.where(fine[..., None], codes, 0)
    return codes.reshape(x.shape).astype(np.uint8), np.where(fine, scale, 0x7F).astype(np.uint8)


def append(codes, scales, x, unit, slots):
    """x [rows, heads, dim] into codes and scales (in place); the later row of one slot counts."""
    new, sc = quantise(x, unit)
    for t, slot in enumerate(slots):
        if 0 <= slot < codes.shape[0] * PAGE:
            codes[slot // PAGE, :, slot % PAGE] = new[t]
            scales[slot // PAGE, :, slot % PAGE] = sc[t]


def logprobs(z, tokens, top, inv_temperature):
    """(logprob, entropy, ids, logprobs) of logits z [rows, n] (FP16), row by row."""
    rows, n = z.shape
    out = np.full(rows, np.nan), np.full(rows, np.nan), np.full((rows, top), -1), np.full((rows, top), np.nan)
    for r in range(rows):
        x = z[r].astype(np.float64)
        if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
            continue
        best = int(x.argmax())
        y = (x - x[best]) * inv_temperature
        e = np.exp(y)
        rest = np.delete(e, best)
        log_s = np.log1p(np.sort(rest).sum())
        out[1][r] = log_s - (e * np.where(e > 0, y, 0)).sum() / (1 + rest.sum())
        if 0 <= tokens[r] < n:
            out[0][r] = y[tokens[r]] - log_s
        out[2][r] = np.argsort(-(x + 0.0), kind="stable")[:top]
        out[3][r] = y[out[2][r]] - log_s
    return out
