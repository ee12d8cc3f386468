"""The speculative-round ABI without a GPU: exports, sizes, argument checks, and pins of the
references the GPU tests use.  No kernel is launched by any test here."""
import ctypes
import math
import os
import re

import numpy as np
import pytest

import kv_ref
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qpn_kv.h")
P = 1 << 20          # a well-aligned address; argument checks never follow it
NULL, SHAPE, ALIGN, BUFFER = 1, 2, 3, 4


@pytest.fixture(scope="module")
def kv():
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def test_every_declared_symbol_is_exported(kv):
    names = sorted(set(re.findall(r"QPN_API\s+[\w\s\*]*?\b(qpn_kv_\w+)\s*\(", open(HEADER).read())))
    assert names == sorted(kv.EXPORTED)
    for n in names:
        assert hasattr(kv.lib, n), n
    assert int(re.search(r"#define QPN_KV_PAGE (\d+)", open(HEADER).read()).group(1)) == kv.PAGE
    assert int(re.search(r"#define QPN_KV_SCRATCH_ZEROED (\d+)", open(HEADER).read()).group(1)) == kv.SCRATCH_ZEROED


def cache(kv, k=P, v=P, ks=P, vs=P, pages=10, heads=2, dim=128):
    return ctypes.byref(kv._Cache(k, v, ks, vs, pages, heads, dim))


def test_cache_errors(kv):
    def call(c):
        return kv.lib.qpn_kv_rope_append(c, P, 512 + 512, 0, 4, P, P, 1e-6, P, 64, 0, P, P, P, 512, None)
    assert call(cache(kv)) == 0                      # no rows: nothing to do
    assert call(None) == NULL
    assert call(cache(kv, k=0)) == NULL and call(cache(kv, vs=0)) == NULL
    assert call(cache(kv, v=P + 8)) == ALIGN and call(cache(kv, ks=P + 2)) == ALIGN
    for bad in (dict(pages=0), dict(pages=1 << 25), dict(heads=0), dict(heads=2000), dict(dim=96), dict(dim=0)):
        assert call(cache(kv, **bad)) == SHAPE, bad


def test_append_errors(kv):
    def call(qkv=P, qs=1024, rows=3, hq=4, qw=P, kw=P, eps=1e-6, f=P, rot=64, pos=P, slots=P, out=P, os=512):
        return kv.lib.qpn_kv_rope_append(cache(kv), qkv, qs, rows, hq, qw, kw, eps, f, rot, 0, pos, slots, out, os,
                                         None)
    for bad in (dict(rows=-1), dict(rows=1 << 21), dict(hq=3), dict(hq=0), dict(hq=2 * 65), dict(rot=8), dict(rot=144),
                dict(rot=-16), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(qs=1016), dict(qs=1028),
                dict(os=504), dict(os=516)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(qkv=None), dict(f=None), dict(pos=None), dict(slots=None), dict(out=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(qkv=P + 8), dict(out=P + 2), dict(qw=P + 2), dict(kw=P + 8), dict(pos=P + 2)):
        assert call(**bad) == ALIGN, bad


def test_plan_errors(kv):
    def call(before=P, rows=P, held=P, n=3, table=P, ts=8, width=8, free=P, cap=5, fc=P, rows_cap=9, seq=P, start=P,
             ho=P, fo=P, slots=P, pos=P):
        return kv.lib.qpn_kv_plan_round(before, rows, held, n, table, ts, width, free, cap, fc, rows_cap, seq, start,
                                        ho, fo, slots, pos, None)
    for bad in (dict(n=-1), dict(n=4097), dict(rows_cap=-1), dict(rows_cap=(1 << 20) + 1), dict(width=-1), dict(ts=7),
                dict(cap=-1), dict(width=1 << 25, ts=1 << 25)):
        assert call(**bad) == SHAPE, bad
    for bad in ("before", "rows", "held", "table", "free", "fc", "seq", "start", "ho", "fo", "slots", "pos"):
        assert call(**{bad: None}) == NULL, bad
        assert call(**{bad: P + 2}) == ALIGN, bad


def test_attention_errors(kv):
    def call(q=P, qs=512, y=P, ys=512, hq=4, rows=3, n=2, most=2, start=P, seq=P, table=P, ts=8, width=8, scale=0.1,
             window=0, scratch=P, sb=0):
        return kv.lib.qpn_kv_attention(cache(kv), q, qs, y, ys, hq, rows, n, most, start, seq, table, ts, width, scale,
                                       window, scratch, sb, None)
    assert call(rows=0) == 0 and call(n=0) == 0
    for bad in (dict(rows=-1), dict(n=-1), dict(n=4097), dict(most=-1), dict(hq=3), dict(ts=7), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(window=-1), dict(qs=504),
                dict(qs=516), dict(ys=504), dict(ys=514)):
        assert call(**bad) == SHAPE, bad
    for bad in ("q", "y", "start", "seq", "table"):
        assert call(**{bad: None}) == NULL, bad
    for bad in (dict(q=P + 8), dict(y=P + 4), dict(start=P + 2), dict(seq=P + 1), dict(table=P + 2), dict(scratch=P + 8)):
        assert call(**bad) == ALIGN, bad
    size = kv.attention_scratch_bytes
    assert size(1, 8, 40, 8, 128, 1) == kv.SCRATCH_ZEROED            # too short to be cut
    assert size(1, 8, 40, 8, 128, 100) > kv.SCRATCH_ZEROED
    for bad in ((-1, 8, 40, 8, 128, 9), (1, 8, 40, 7, 128, 9), (1, 8, 40, 8, 96, 9), (1, -1, 40, 8, 128, 9),
                (4097, 8, 40, 8, 128, 9), (1, 8, 40, 8, 128, -1)):
        assert size(*bad) == 2 ** 64 - 1, bad


def test_verify_errors(kv):
    need = kv.verify_scratch_bytes(3, 2, 1000)

    def call(x=P, xs=1000, d=None, ds=0, tok=P, start=P, rows=3, n=2, vocab=1000, it=1.0, u=P, su=P, acc=P, nxt=P,
             prob=P, scratch=P, sb=need):
        return kv.lib.qpn_kv_verify_sampled(x, xs, d, ds, tok, start, rows, n, vocab, it, u, su, acc, nxt, prob,
                                            scratch, sb, None)
    assert call(n=0) == 0
    for bad in (dict(rows=-1), dict(rows=65536), dict(n=-1), dict(n=4097), dict(vocab=0), dict(vocab=(1 << 24) + 1),
                dict(it=0.0), dict(it=-1.0), dict(it=math.nan), dict(it=math.inf), dict(xs=999), dict(d=P, ds=999)):
        assert call(**bad) == SHAPE, bad
    for bad in ("x", "tok", "start", "u", "su", "acc", "nxt", "prob", "scratch"):
        assert call(**{bad: None}) == NULL, bad
    for bad in (dict(x=P + 1), dict(d=P + 1, ds=1000), dict(tok=P + 2), dict(start=P + 2), dict(prob=P + 1),
                dict(scratch=P + 8)):
        assert call(**bad) == ALIGN, bad
    assert call(sb=need - 1) == BUFFER
    assert kv.verify_scratch_bytes(-1, 1, 10) == kv.verify_scratch_bytes(1, 1, 0) == 2 ** 64 - 1


def test_valid_call_without_gpu_reports_device_error(kv):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert kv.lib.qpn_kv_attention(cache(kv), P, 512, P, 512, 4, 3, 2, 2, P, P, P, 8, 8, 0.1, 0, P, 0, None) == 5


def test_binding_refuses_wrong_tensors(kv):
    import torch
    cpu = torch.zeros(4, 1024, dtype=torch.float16)
    with pytest.raises(ValueError):
        kv.KvCache.empty(2, 2, 128, device="cpu")
    with pytest.raises(ValueError):
        kv._rows(cpu, "x")
    with pytest.raises(ValueError):
        kv._need(cpu, torch.int32, 2, "x")
    with pytest.raises(ValueError):
        kv._table(torch.zeros(2, 3, dtype=torch.int32), 2)


# ---------------------------------------------------------------- the references

def test_reference_codes_are_the_oracles():
    # the oracle states the format on its own; float8_e4m3fn is a third statement
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(t), np.isnan(kv_ref.VALUES))
    ok = ~np.isnan(t)
    assert np.array_equal(t[ok], kv_ref.VALUES[ok])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.integers(-4, 3, 4000), kv_ref.VALUES[ok],
                        (kv_ref.VALUES[:126] + kv_ref.VALUES[1:127]) / 2])
    x = np.clip(x, -448, 448).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, kv_ref.e4m3_codes(x.astype(np.float64)))


def test_reference_layout_round_trips():
    c = np.random.default_rng(1).integers(0, 256, (3, 2, 64, 64)).astype(np.uint8)
    assert np.array_equal(kv_ref.unpack_k(kv_ref.pack_k(c)), c)
    assert np.array_equal(kv_ref.unpack_v(kv_ref.pack_v(c)), c)
    assert kv_ref.pack_k(c)[1, 0, 2, 30, 5] == c[1, 0, 30, 37]
    # token 16 t + 4 g + r = 39: t 2, g 1, r 3, at 16 g + 4 t + r = 27
    assert kv_ref.pack_v(c)[2, 1, 9, 27] == c[2, 1, 39, 9]


def test_reference_page_scale():
    assert kv_ref.page_scale(448.0) == 1.0 and kv_ref.page_scale(448.0001) == 2.0
    assert kv_ref.page_scale(0.0) == 2.0 ** -60 and kv_ref.page_scale(1.75) == 2.0 ** -8


def test_reference_verify_worked_example():
    # two tokens of probability 3/4 and 1/4 against a drafter's 1/4 and 3/4: the
    # draft 1 is accepted with probability 1/3, else token 0 is the only one left
    lp, lq = np.log([[0.75, 0.25], [0.75, 0.25]]), np.log([[0.25, 0.75], [0.25, 0.75]])
    for u, want in ((0.3, ([1], [0])), (0.34, ([0], [0]))):
        acc, nxt, prob = kv_ref.verify(lp, lq, [0, 1], [0, 2], 1.0, [u, 0], [0.5])
        assert (acc, nxt) == want and abs(prob[0] - 1 / 3) < 1e-12
    assert kv_ref.verify(lp, lq, [0, 1], [0, 2], 1.0, [0.3, 0], [0.76])[1] == [1]
    # a greedy drafter: accepted with probability 1/4; refused, only token 0 remains
    assert kv_ref.verify(lp, None, [0, 1], [0, 2], 1.0, [0.26, 0], [0.99])[:2] == ([0], [0])
