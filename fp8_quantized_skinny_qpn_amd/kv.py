"""Thin ctypes binding of the speculative-round operators (the C ABI in include/qpn_kv.h).

The operators around the packed-weight products of ``qpn``: page tables of a round, the cache
append with query/key norms and rotation, attention over an 8-bit paged KV cache or a 4-bit one
(include/qpn_kv4.h), reading the latter's tokens back, the verification of sampled drafts, and log
probabilities.  As in ``qpn``, argument marshalling only: every step of the
computation runs in the HIP kernels of libqpn.so, and there is no fallback of any kind.

One round, on the device throughout::

    r = kv.plan_round(before, rows, held, table, free_pages, free_count, capacity)
    qkv = qpn.gemm(w_qkv, x)
    q = kv.rope_append(cache, qkv, q_heads, r.positions, r.slots, inv_freq, q_weight, k_weight)
    y = kv.attention(cache, q, r.row_start, r.seq_lens, table, max_rows)
    ...                                    # O, gate/up, down, lm_head
    accepted, token, prob = kv.verify_sampled(logits, tokens, r.row_start, accept_u, sample_u)
    logprob, entropy, ids, logprobs = kv.logprobs(logits, drafts, top=5)   # what a server answers with

Attention, verification and log probabilities pass sums on through a scratch that calls on one stream share, from any
thread; calls captured into a graph share one of the graph's own, so graphs may run beside each
other and beside calls.  A call may be given a scratch (`scratch_`, uint8): its first SCRATCH_ZEROED
bytes zero before the first use, and no two calls at a time.
"""
import ctypes
from contextlib import nullcontext
from dataclasses import dataclass
from functools import lru_cache

import torch

from .qpn import StreamBuffers, _empty, _torch_stream, check, lib

PAGE = 64
SCRATCH_ZEROED = 65536
MAX_TOP = 32


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32)]


class _Cache4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "k_unit", "v_unit")] + [
        ("pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


def _bind():
    c = ctypes
    vp, i64, sz, i32, f64, f32 = c.c_void_p, c.c_int64, c.c_size_t, c.c_int, c.c_double, c.c_float
    cp = c.POINTER(_Cache)
    sig = {
        "qpn_kv_plan_round": ([vp, vp, vp, i32, vp, i64, i32, vp, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp], i32),
        "qpn_kv_rope_append": ([cp, vp, i64, i32, i32, vp, vp, f64, vp, i32, i32, vp, vp, vp, i64, vp], i32),
        "qpn_kv_attention_scratch_bytes": ([i32, i32, i32, i32, i32, i32], sz),
        "qpn_kv_attention": ([cp, vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp, i64, i32, f32, i32, vp, sz, vp],
                             i32),
        "qpn_kv_verify_scratch_bytes": ([i32, i32, i64], sz),
        "qpn_kv_verify_sampled": ([vp, i64, vp, i64, vp, vp, i32, i32, i64, f64, vp, vp, vp, vp, vp, vp, sz, vp],
                                  i32),
        "qpn_kv_logprobs_scratch_bytes": ([i32, i64], sz),
        "qpn_kv_logprobs": ([vp, i64, vp, i32, i64, f64, i32, vp, vp, vp, vp, vp, sz, vp], i32),
    }
    sig4 = {
        "qpn_kv4_read": ([c.POINTER(_Cache4), vp, i32, vp, i64, vp, i64, vp], i32),
    }
    for name in ("rope_append", "attention_scratch_bytes", "attention"):
        args, res = sig["qpn_kv_" + name]
        sig4["qpn_kv4_" + name] = ([c.POINTER(_Cache4) if t is cp else t for t in args], res)
    for name, (args, res) in (*sig.items(), *sig4.items()):
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return tuple(sig), tuple(sig4)


# Symbols the C headers declare (qpn_kv.h, qpn_kv4.h).
EXPORTED, EXPORTED4 = _bind()


def _need(t, dtype, dim, what):
    """A contiguous device tensor of this type and rank."""
    if t.dtype is dtype and t.is_cuda and t.dim() == dim and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous {dim}-D {dtype} CUDA tensor")


def _rows(t, what):
    """(pointer, row stride) of FP16 rows: unit stride within a row."""
    if t.dtype is torch.float16 and t.is_cuda and t.dim() == 2:
        (n, width), (stride, step) = t.shape, t.stride()
        if step == 1 or width == 1:
            return t.data_ptr(), stride if n > 1 else max(width, 1)
    raise ValueError(f"{what} must be a 2-D float16 CUDA tensor with unit stride in its rows")


def _table(t, requests):
    if not (t.dtype is torch.int32 and t.is_cuda and t.dim() == 2):
        raise ValueError("the page table must be a 2-D int32 CUDA tensor with unit stride in its rows")
    (n, width), (stride, step) = t.shape, t.stride()
    if not (step == 1 or width <= 1 or n == 0):
        raise ValueError("the page table must be a 2-D int32 CUDA tensor with unit stride in its rows")
    if n != requests:
        raise ValueError(f"the page table has {n} rows for {requests} requests")
    return t.data_ptr(), stride if n > 1 and width else max(width, 1), width


def _raw_stream(stream) -> int:
    """The HIP stream of a call: the given torch stream's, else the current device's current one.
    (torch.cuda.current_stream() builds an object, which costs more than the rest of a call.)"""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


# Scratch of attention, verification and log probabilities: its zeroed head is left zero by every
# call, the rest holds anything.  A call of several launches passes its sums on
# through the scratch, so a call holds its scratch's lock until all of them are
# queued: threads that share a stream queue whole calls one after another.
_buffers = StreamBuffers(SCRATCH_ZEROED, SCRATCH_ZEROED)
_scratches, _locks = _buffers.held, _buffers.locks
_unlocked = nullcontext()  # for a call that is given its scratch


class KvCache:
    """One layer's cache: pages of 64 tokens, E4M3 codes with a scale per page and head.

    k: float8_e4m3fn [pages, heads, dim / 16, 64, 16]: dimension 16 c + e of token t at [c, t, e];
    v: float8_e4m3fn [pages, heads, dim, 64]: dimension d of token 16 t + 4 g + r at
    [d, 16 g + 4 t + r]; k_scale, v_scale: float32 [pages, heads].  Setting a field (a cache that
    grows) takes effect at the next call, which checks them all."""

    def __init__(self, k, v, k_scale, v_scale):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self._checked()

    def __setattr__(self, name, value):
        if name == "k":
            if value.dim() != 5 or value.shape[3] != PAGE or value.shape[4] != 16:
                raise ValueError("keys must be [pages, heads, dim / 16, 64, 16]")
            self.__dict__.update(pages=value.shape[0], heads=value.shape[1], dim=value.shape[2] * 16)
        self.__dict__["_ref"] = None
        self.__dict__[name] = value

    def _checked(self):
        """The C struct of the tensors, checked once after a field is set."""
        if self._ref is None:
            pages, heads, dim, f8, f32 = self.pages, self.heads, self.dim, torch.float8_e4m3fn, torch.float32
            if tuple(self.v.shape) != (pages, heads, dim, PAGE):
                raise ValueError("values must be [pages, heads, dim, 64]")
            if tuple(self.k_scale.shape) != (pages, heads) or tuple(self.v_scale.shape) != (pages, heads):
                raise ValueError("scales must be [pages, heads]")
            self.__dict__["_ref"] = ctypes.byref(_Cache(
                _need(self.k, f8, 5, "keys"), _need(self.v, f8, 4, "values"), _need(self.k_scale, f32, 2, "key scales"),
                _need(self.v_scale, f32, 2, "value scales"), pages, heads, dim))
        return self._ref

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, device="cuda") -> "KvCache":
        """A cache of pages no request holds yet."""
        f8 = torch.float8_e4m3fn
        return cls(torch.zeros((pages, heads, dim // 16, PAGE, 16), dtype=f8, device=device),
                   torch.zeros((pages, heads, dim, PAGE), dtype=f8, device=device),
                   torch.ones((pages, heads), device=device), torch.ones((pages, heads), device=device))


    _append, _attention = "qpn_kv_rope_append", "qpn_kv_attention"

    @staticmethod
    def _scratch_bytes(*sizes):
        return attention_scratch_bytes(*sizes)


class KvCache4(KvCache):
    """One layer's cache in 4 bits: pages of 64 tokens, E2M1 codes with an E4M3 scale per token, head and
    16 dimensions, and a float32 unit per head (a value is code * scale * unit; layout: include/qpn_kv4.h).

    k, v: uint8 [pages, heads, dim / 32, 64, 16]; k_scale: float8_e4m3fn [pages, heads, 64, dim / 16];
    v_scale: float8_e4m3fn [pages, heads, dim / 64, 16, 16]; k_unit, v_unit: float32 [heads], positive:
    2688 units are the largest value, and a group whose largest is below 0.09 units has a coarser scale.
    Setting a field takes effect at the next call."""

    def __init__(self, k, v, k_scale, v_scale, k_unit, v_unit):
        self.k_unit, self.v_unit = k_unit, v_unit
        super().__init__(k, v, k_scale, v_scale)

    def __setattr__(self, name, value):
        if name == "k":
            if value.dim() != 5 or value.shape[3] != PAGE or value.shape[4] != 16:
                raise ValueError("keys must be [pages, heads, dim / 32, 64, 16]")
            self.__dict__.update(pages=value.shape[0], heads=value.shape[1], dim=value.shape[2] * 32)
        self.__dict__["_ref"] = None
        self.__dict__[name] = value

    def _checked(self):
        if self._ref is None:
            pages, heads, dim = self.pages, self.heads, self.dim
            u8, f8, f32 = torch.uint8, torch.float8_e4m3fn, torch.float32
            if self.v.shape != self.k.shape:
                raise ValueError("values must have the keys' shape")
            if tuple(self.k_scale.shape) != (pages, heads, PAGE, dim // 16) \
                    or tuple(self.v_scale.shape) != (pages, heads, dim // 64, 16, 16):
                raise ValueError("scales must be [pages, heads, 64, dim / 16] and [pages, heads, dim / 64, 16, 16]")
            if tuple(self.k_unit.shape) != (heads,) or tuple(self.v_unit.shape) != (heads,):
                raise ValueError("units must be [heads]")
            self.__dict__["_ref"] = ctypes.byref(_Cache4(
                _need(self.k, u8, 5, "keys"), _need(self.v, u8, 5, "values"), _need(self.k_scale, f8, 4, "key scales"),
                _need(self.v_scale, f8, 5, "value scales"), _need(self.k_unit, f32, 1, "key units"),
                _need(self.v_unit, f32, 1, "value units"), pages, heads, dim))
        return self._ref

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, device="cuda", unit: float = 0.125) -> "KvCache4":
        """A cache of pages no request holds yet."""
        z = lambda dtype, *s: torch.zeros((pages, heads) + s, dtype=torch.uint8, device=device).view(dtype)  # noqa: E731
        u8, f8 = torch.uint8, torch.float8_e4m3fn
        return cls(z(u8, dim // 32, PAGE, 16), z(u8, dim // 32, PAGE, 16), z(f8, PAGE, dim // 16),
                   z(f8, dim // 64, 16, 16), torch.full((heads,), unit, dtype=torch.float32, device=device),
                   torch.full((heads,), unit, dtype=torch.float32, device=device))

    _append, _attention = "qpn_kv4_rope_append", "qpn_kv4_attention"

    @staticmethod
    def _scratch_bytes(*sizes):
        return attention4_scratch_bytes(*sizes)


@dataclass
class Round:
    """What plan_round writes: int32 device tensors."""
    seq_lens: torch.Tensor    # [requests]
    row_start: torch.Tensor   # [requests + 1]
    held: torch.Tensor        # [requests]
    free_count: torch.Tensor  # [1]
    slots: torch.Tensor       # [capacity]
    positions: torch.Tensor   # [capacity]

    @classmethod
    def empty(cls, requests: int, capacity: int, device="cuda") -> "Round":
        e = lambda n: torch.empty(n, dtype=torch.int32, device=device)  # noqa: E731
        return cls(e(requests), e(requests + 1), e(requests), e(1), e(capacity), e(capacity))

    def __setattr__(self, name, value):
        self.__dict__["_args"] = None
        self.__dict__[name] = value

    def _checked(self):
        """(requests, capacity, the six pointers), checked once after a field is set."""
        if self._args is None:
            n, cap = self.seq_lens.shape[0], self.slots.shape[0]
            if self.held.shape[0] != n or self.row_start.shape[0] != n + 1 \
                    or self.positions.shape[0] != cap or self.free_count.numel() != 1:
                raise ValueError("sizes of the requests' tensors do not agree")
            self.__dict__["_args"] = (n, cap) + tuple(
                _need(getattr(self, k), torch.int32, 1, k)
                for k in ("seq_lens", "row_start", "held", "free_count", "slots", "positions"))
        return self._args


def plan_round(before, rows, held, table, free_pages, free_count, capacity: int = None, out: Round = None,
               stream=None) -> Round:
    """Page tables, row_start, slots and positions of a round through qpn_kv_plan_round; the
    table's new entries are written in place.  `capacity` (rows) or `out` is needed."""
    i32 = torch.int32
    n = before.shape[0]
    if out is None:
        if capacity is None:
            raise ValueError("capacity or out is needed")
        with torch.cuda.stream(_torch_stream(stream)):
            out = Round.empty(n, capacity, before.device)
    requests, cap, seq_p, start_p, held_p, count_p, slots_p, pos_p = out._checked()
    if capacity is not None and capacity != cap:
        raise ValueError(f"out has room for {cap} rows, not {capacity}")
    if requests != n or rows.shape[0] != n or held.shape[0] != n or free_count.numel() != 1:
        raise ValueError("sizes of the requests' tensors do not agree")
    tp, tstride, width = _table(table, n)
    check(lib.qpn_kv_plan_round(
        _need(before, i32, 1, "before"), _need(rows, i32, 1, "rows"), _need(held, i32, 1, "held"), n, tp, tstride,
        width, _need(free_pages, i32, 1, "free_pages"), free_pages.shape[0], _need(free_count, i32, 1, "free_count"),
        cap, seq_p, start_p, held_p, count_p, slots_p, pos_p, _raw_stream(stream)))
    return out


def rope_append(cache: KvCache, qkv, q_heads: int, positions, slots, inv_freq, q_weight=None, k_weight=None,
                eps: float = 1e-6, interleaved: bool = False, out=None, stream=None) -> torch.Tensor:
    """Norms, rotation and cache append of QKV rows through qpn_kv_rope_append (qpn_kv4_rope_append
    for a KvCache4); returns the queries
    [rows, q_heads * dim].  inv_freq: float32 [rot / 2] (None: no rotation)."""
    d = cache.dim
    rows = qkv.shape[0]
    qp, qs = _rows(qkv, "qkv")
    if qkv.shape[1] != (q_heads + 2 * cache.heads) * d:
        raise ValueError(f"qkv has {qkv.shape[1]} columns for {q_heads} + 2 * {cache.heads} heads of {d}")
    if positions.shape[0] != rows or slots.shape[0] != rows:
        raise ValueError("positions and slots must have one entry per row")
    for w in (q_weight, k_weight):
        if w is not None and w.shape[0] != d:
            raise ValueError(f"norm weights must have {d} elements")
    if out is None:
        out = _empty(_torch_stream(stream), (rows, q_heads * d), torch.float16, qkv.device)
    op, os = _rows(out, "out")
    if tuple(out.shape) != (rows, q_heads * d):
        raise ValueError(f"out must be [{rows}, {q_heads * d}]")
    f16, i32 = torch.float16, torch.int32
    check(getattr(lib, cache._append)(
        cache._ref or cache._checked(), qp, qs, rows, q_heads,
        None if q_weight is None else _need(q_weight, f16, 1, "q_weight"),
        None if k_weight is None else _need(k_weight, f16, 1, "k_weight"), eps,
        None if inv_freq is None else _need(inv_freq, torch.float32, 1, "inv_freq"),
        0 if inv_freq is None else 2 * inv_freq.shape[0], interleaved, _need(positions, i32, 1, "positions"),
        _need(slots, i32, 1, "slots"), op, os, _raw_stream(stream)))
    return out


def read(cache: KvCache4, slots, out=None, stream=None):
    """(keys, values) float16 [rows, heads * dim] of the tokens slots [rows] through qpn_kv4_read: what the
    cache holds for them; zeros for a slot outside the cache."""
    if not isinstance(cache, KvCache4):
        raise TypeError("tokens are read back from a KvCache4")
    rows, width = slots.shape[0], cache.heads * cache.dim
    sp = _need(slots, torch.int32, 1, "slots")
    if out is None:
        ts = _torch_stream(stream)
        out = (_empty(ts, (rows, width), torch.float16, slots.device),
               _empty(ts, (rows, width), torch.float16, slots.device))
    k, v = out
    if tuple(k.shape) != (rows, width) or tuple(v.shape) != (rows, width):
        raise ValueError(f"out must be two of [{rows}, {width}]")
    (kp, ks), (vp, vs) = _rows(k, "out"), _rows(v, "out")
    check(lib.qpn_kv4_read(cache._ref or cache._checked(), sp, rows, kp, ks, vp, vs, _raw_stream(stream)))
    return out


@lru_cache(maxsize=1024)
def attention_scratch_bytes(requests: int, max_rows: int, q_heads: int, heads: int, dim: int, width: int) -> int:
    return int(lib.qpn_kv_attention_scratch_bytes(requests, max_rows, q_heads, heads, dim, width))


@lru_cache(maxsize=1024)
def attention4_scratch_bytes(requests: int, max_rows: int, q_heads: int, heads: int, dim: int, width: int) -> int:
    return int(lib.qpn_kv4_attention_scratch_bytes(requests, max_rows, q_heads, heads, dim, width))


def attention(cache: KvCache, q, row_start, seq_lens, table, max_rows: int, scale: float = None, window: int = 0,
              out=None, stream=None, scratch_=None) -> torch.Tensor:
    """Attention of the rows q [rows, q_heads * dim] over the cache through qpn_kv_attention
    (qpn_kv4_attention for a KvCache4).
    `max_rows`: the most rows of one request (a hint; over a KvCache4 the table's width is one of its
    length).  `scale` defaults to dim ** -0.5."""
    d = cache.dim
    n = seq_lens.shape[0]
    shape = q.shape
    if len(shape) != 2 or shape[1] % d:
        raise ValueError(f"queries must be [rows, heads * {d}]")
    if row_start.shape[0] != n + 1:
        raise ValueError("row_start must have one entry more than seq_lens")
    heads = shape[1] // d
    qp, qs = _rows(q, "queries")
    tp, tstride, width = _table(table, n)
    raw = _raw_stream(stream)
    if out is None:
        out = _empty(_torch_stream(stream), tuple(shape), torch.float16, q.device)
    elif out.shape != shape:
        raise ValueError("out must have the queries' shape")
    yp, ys = _rows(out, "out")
    key = (q.get_device(), raw)
    with _locks[key] if scratch_ is None else _unlocked:
        if scratch_ is None:
            need = cache._scratch_bytes(n, max_rows, heads, cache.heads, d, width)
            scratch_ = _buffers.get(need if need < 1 << 63 else 0, key, stream)
        else:
            _need(scratch_, torch.uint8, 1, "scratch_")
        check(getattr(lib, cache._attention)(
            cache._ref or cache._checked(), qp, qs, yp, ys, heads, shape[0], n, max_rows,
            _need(row_start, torch.int32, 1, "row_start"), _need(seq_lens, torch.int32, 1, "seq_lens"), tp, tstride,
            width, d ** -0.5 if scale is None else scale, window, scratch_.data_ptr(), scratch_.numel(), raw))
    return out


@lru_cache(maxsize=1024)
def verify_scratch_bytes(rows: int, requests: int, n: int) -> int:
    return int(lib.qpn_kv_verify_scratch_bytes(rows, requests, n))


def verify_sampled(logits, tokens, row_start, accept_u, sample_u, draft_logits=None, temperature: float = 1.0,
                   out=None, stream=None, scratch_=None):
    """(accepted int32 [requests], next int32 [requests], accept_prob float32 [rows]) through
    qpn_kv_verify_sampled.  draft_logits None: a greedy drafter."""
    rows, n = logits.shape
    requests = row_start.shape[0] - 1
    lp, ls = _rows(logits, "logits")
    dp = ds = 0
    if draft_logits is not None:
        dp, ds = _rows(draft_logits, "draft_logits")
        if draft_logits.shape != logits.shape:
            raise ValueError("draft_logits must have the logits' shape")
    if tokens.shape[0] != rows or accept_u.shape[0] != rows or sample_u.shape[0] != requests:
        raise ValueError("tokens and accept_u need one entry per row, sample_u one per request")
    if not temperature > 0:
        raise ValueError("temperature must be positive")
    raw = _raw_stream(stream)
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if out is None:
        ts = _torch_stream(stream)
        out = (_empty(ts, (requests,), i32, dev), _empty(ts, (requests,), i32, dev), _empty(ts, (rows,), f32, dev))
    accepted, token, prob = out
    if accepted.shape[0] != requests or token.shape[0] != requests or prob.shape[0] != rows:
        raise ValueError("out must be (accepted [requests], next [requests], accept_prob [rows])")
    key = (logits.get_device(), raw)
    with _locks[key] if scratch_ is None else _unlocked:
        if scratch_ is None:
            need = verify_scratch_bytes(rows, requests, n)
            scratch_ = _buffers.get(need if need < 1 << 63 else 0, key, stream)
        else:
            _need(scratch_, torch.uint8, 1, "scratch_")
        check(lib.qpn_kv_verify_sampled(
            lp, ls, dp or None, ds, _need(tokens, i32, 1, "tokens"), _need(row_start, i32, 1, "row_start"), rows,
            requests, n, 1.0 / temperature, _need(accept_u, f32, 1, "accept_u"),
            _need(sample_u, f32, 1, "sample_u"), _need(accepted, i32, 1, "accepted"), _need(token, i32, 1, "next"),
            _need(prob, f32, 1, "accept_prob"), scratch_.data_ptr(), scratch_.numel(), raw))
    return out


@lru_cache(maxsize=1024)
def logprobs_scratch_bytes(rows: int, n: int) -> int:
    return int(lib.qpn_kv_logprobs_scratch_bytes(rows, n))


def logprobs(logits, tokens, top: int = 0, temperature: float = 1.0, out=None, stream=None, scratch_=None):
    """(logprob float32 [rows], entropy float32 [rows], top_ids int32 [rows, top], top_logprobs float32
    [rows, top]) through qpn_kv_logprobs: the log probabilities of tokens [rows] under
    softmax(logits / temperature), its entropy, and the likeliest tokens (equal ones: the lowest first)."""
    rows, n = logits.shape
    lp, ls = _rows(logits, "logits")
    if tokens.shape[0] != rows:
        raise ValueError("tokens must have one entry per row")
    if not temperature > 0:
        raise ValueError("temperature must be positive")
    if not 0 <= top <= min(n, MAX_TOP):
        raise ValueError(f"top must be from 0 to {min(n, MAX_TOP)}")
    raw = _raw_stream(stream)
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    if out is None:
        ts = _torch_stream(stream)
        out = (_empty(ts, (rows,), f32, dev), _empty(ts, (rows,), f32, dev), _empty(ts, (rows, top), i32, dev),
               _empty(ts, (rows, top), f32, dev))
    logprob, entropy, ids, alternatives = out
    if logprob.shape[0] != rows or entropy.shape[0] != rows or tuple(ids.shape) != (rows, top) \
            or tuple(alternatives.shape) != (rows, top):
        raise ValueError("out must be (logprob [rows], entropy [rows], top_ids [rows, top], top_logprobs [rows, top])")
    key = (logits.get_device(), raw)
    with _locks[key] if scratch_ is None else _unlocked:
        if scratch_ is None:
            need = logprobs_scratch_bytes(rows, n)
            scratch_ = _buffers.get(need if need < 1 << 63 else 0, key, stream)
        else:
            _need(scratch_, torch.uint8, 1, "scratch_")
        check(lib.qpn_kv_logprobs(
            lp, ls, _need(tokens, i32, 1, "tokens"), rows, n, 1.0 / temperature, top,
            _need(logprob, f32, 1, "logprob"), _need(entropy, f32, 1, "entropy"), _need(ids, i32, 2, "top_ids"),
            _need(alternatives, f32, 2, "top_logprobs"), scratch_.data_ptr(), scratch_.numel(), raw))
    return out
