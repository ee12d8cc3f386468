"""The 4-bit cache and the log probabilities without a GPU: exports, sizes, argument checks, and pins of
the references the GPU tests use.  No kernel is launched by any test here."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import kv4_ref
import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qpn_kv4.h")
P = 1 << 20          # a well-aligned address; argument checks never follow it
NULL, SHAPE, ALIGN, BUFFER, DEVICE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def kv():
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def cache(kv, k=P, v=P, ks=P, vs=P, ku=P, vu=P, pages=10, heads=2, dim=128):
    return ctypes.byref(kv._Cache4(k, v, ks, vs, ku, vu, pages, heads, dim))


def test_every_declared_symbol_is_exported(kv):
    names = sorted(set(re.findall(r"QPN_API\s+[\w\s\*]*?\b(qpn_kv4_\w+)\s*\(", open(HEADER).read())))
    assert names == sorted(kv.EXPORTED4)
    for n in names:
        assert hasattr(kv.lib, n), n
    head = open(os.path.join(ROOT, "include", "qpn_kv.h")).read()
    assert int(re.search(r"#define QPN_KV_MAX_TOP (\d+)", head).group(1)) == kv.MAX_TOP


def test_cache_errors(kv):
    calls = [lambda c: kv.lib.qpn_kv4_rope_append(c, P, 1024, 0, 4, P, P, 1e-6, P, 64, 0, P, P, P, 512, None),
             lambda c: kv.lib.qpn_kv4_read(c, P, 0, P, 2048, P, 2048, None),
             lambda c: kv.lib.qpn_kv4_attention(c, P, 512, P, 512, 4, 0, 1, 1, P, P, P, 8, 8, 0.1, 0, P, 0, None)]
    for call in calls:
        assert call(None) == NULL
        for bad in (dict(k=0), dict(v=0), dict(ks=0), dict(vs=0), dict(ku=0), dict(vu=0)):
            assert call(cache(kv, **bad)) == NULL, bad
        for bad in (dict(k=P + 8), dict(v=P + 4), dict(ks=P + 8), dict(vs=P + 1), dict(ku=P + 2), dict(vu=P + 1)):
            assert call(cache(kv, **bad)) == ALIGN, bad
        for bad in (dict(pages=0), dict(pages=1 << 25), dict(heads=0), dict(heads=2000), dict(dim=96), dict(dim=0)):
            assert call(cache(kv, **bad)) == SHAPE, bad
    assert calls[0](cache(kv)) == 0 and calls[1](cache(kv, heads=8, dim=256)) == 0 and calls[2](cache(kv)) == 0


def test_append_errors(kv):
    def call(qkv=P, qs=1024, rows=3, hq=4, qw=P, kw=P, eps=1e-6, f=P, rot=64, pos=P, slots=P, out=P, os=512):
        return kv.lib.qpn_kv4_rope_append(cache(kv), qkv, qs, rows, hq, qw, kw, eps, f, rot, 0, pos, slots, out, os, None)
    for bad in (dict(rows=-1), dict(rows=1 << 21), dict(hq=3), dict(hq=0), dict(hq=2 * 65), dict(rot=8), dict(rot=144),
                dict(rot=-16), dict(eps=-1.0), dict(eps=math.nan), dict(qs=1016), dict(qs=1028), dict(os=504), dict(os=516)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(qkv=None), dict(f=None), dict(pos=None), dict(slots=None), dict(out=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(qkv=P + 8), dict(out=P + 2), dict(qw=P + 2), dict(kw=P + 8), dict(pos=P + 2), dict(slots=P + 1)):
        assert call(**bad) == ALIGN, bad


def test_read_errors(kv):
    def call(slots=P, rows=3, k=P, ks=256, v=P, vs=256, **c):
        return kv.lib.qpn_kv4_read(cache(kv, **c), slots, rows, k, ks, v, vs, None)
    for bad in (dict(rows=-1), dict(rows=1 << 21), dict(ks=248), dict(vs=248), dict(ks=260), dict(vs=257),
                dict(rows=1 << 20, heads=64, ks=8192, vs=8192)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(slots=None), dict(k=None), dict(v=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(slots=P + 2), dict(k=P + 8), dict(v=P + 2)):
        assert call(**bad) == ALIGN, bad
    if not torch.cuda.is_available():
        assert call() == DEVICE


def test_attention_errors(kv):
    def call(q=P, qs=512, y=P, ys=512, hq=4, rows=3, requests=1, most=3, start=P, seq=P, table=P, ts=8, width=8, scale=0.1,
             window=0, scratch=P, nbytes=1 << 20):
        return kv.lib.qpn_kv4_attention(cache(kv), q, qs, y, ys, hq, rows, requests, most, start, seq, table, ts, width,
                                        scale, window, scratch, nbytes, None)
    for bad in (dict(rows=-1), dict(requests=5000), dict(most=-1), dict(hq=5), dict(width=1 << 25), dict(ts=7), dict(scale=0.0),
                dict(scale=math.inf), dict(scale=math.nan), dict(window=-1), dict(qs=504), dict(qs=516), dict(ys=510)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(q=None), dict(y=None), dict(start=None), dict(seq=None), dict(table=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(q=P + 8), dict(y=P + 4), dict(start=P + 2), dict(seq=P + 1), dict(table=P + 2), dict(scratch=P + 8)):
        assert call(**bad) == ALIGN, bad
    bytes_of = kv.lib.qpn_kv4_attention_scratch_bytes
    for bad in ((-1, 1, 4, 2, 128, 8), (1, -1, 4, 2, 128, 8), (1, 1, 5, 2, 128, 8), (1, 1, 4, 2, 96, 8), (1, 1, 4, 2, 128, -1)):
        assert bytes_of(*bad) == ctypes.c_size_t(-1).value
    assert bytes_of(1, 8, 40, 8, 128, 8) == kv.SCRATCH_ZEROED < bytes_of(1, 8, 40, 8, 128, 9)


def test_logprobs_errors(kv):
    def call(z=P, zs=100, tokens=P, rows=2, n=100, inv=1.0, top=5, lp=P, h=P, ids=P, lps=P, scratch=P, nbytes=1 << 24):
        return kv.lib.qpn_kv_logprobs(z, zs, tokens, rows, n, inv, top, lp, h, ids, lps, scratch, nbytes, None)
    for bad in (dict(rows=-1), dict(rows=65536), dict(n=0), dict(n=(1 << 24) + 1, zs=1 << 25), dict(zs=99), dict(inv=0.0),
                dict(inv=-1.0), dict(inv=math.inf), dict(inv=math.nan), dict(top=-1), dict(top=33), dict(n=4, top=5)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(z=None), dict(tokens=None), dict(lp=None), dict(h=None), dict(ids=None), dict(lps=None), dict(scratch=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(z=P + 1), dict(tokens=P + 2), dict(lp=P + 1), dict(h=P + 2), dict(ids=P + 2), dict(lps=P + 1),
                dict(scratch=P + 8)):
        assert call(**bad) == ALIGN, bad
    assert call(nbytes=100) == BUFFER
    assert call(rows=0) == 0
    size = kv.lib.qpn_kv_logprobs_scratch_bytes
    assert size(-1, 5) == size(1, 0) == size(65536, 5) == size(1, (1 << 24) + 1) == ctypes.c_size_t(-1).value
    assert size(1, 100) == size(65535, 1 << 24) == kv.SCRATCH_ZEROED < size(1, 151936) < size(8, 151936) < 1 << 24
    if not torch.cuda.is_available():
        assert call() == DEVICE and call(ids=None, lps=None, top=0) == DEVICE


def test_binding_refuses(kv):
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    h = lambda *n: torch.zeros(*n, dtype=torch.float16)  # noqa: E731
    with pytest.raises(ValueError):
        kv.KvCache4.empty(2, 2, 64, device="cpu")                     # host tensors
    with pytest.raises(TypeError):
        kv.read(object.__new__(kv.KvCache), i(3))
    with pytest.raises(ValueError, match="logits"):
        kv.logprobs(h(3, 9), i(3))                                    # host logits
    with pytest.raises(ValueError, match="logits"):
        kv.logprobs(torch.zeros(3, 9), i(3))


def test_cache_follows_its_fields(kv, monkeypatch):
    def need(t, dtype, dim, what):
        if t.dtype is dtype and t.dim() == dim and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(what)
    monkeypatch.setattr(kv, "_need", need)
    new = lambda pages, heads=2, dim=64: kv.KvCache4.empty(pages, heads, dim, device="cpu")  # noqa: E731
    struct = lambda c: ctypes.cast(c._checked(), ctypes.POINTER(kv._Cache4)).contents  # noqa: E731
    c, wide = new(3), new(5, 3, 256)
    s = struct(c)
    assert (s.pages, s.heads, s.dim) == (3, 2, 64) == (c.pages, c.heads, c.dim)
    c.k = wide.k
    with pytest.raises(ValueError, match="values"):
        struct(c)
    c.v = wide.v
    with pytest.raises(ValueError, match="scales"):
        struct(c)
    c.k_scale, c.v_scale = wide.k_scale, wide.v_scale
    with pytest.raises(ValueError, match="units"):
        struct(c)
    c.k_unit, c.v_unit = wide.k_unit, wide.v_unit
    s = struct(c)
    assert (s.pages, s.heads, s.dim) == (5, 3, 256)
    names = ("k", "v", "k_scale", "v_scale", "k_unit", "v_unit")
    assert [getattr(s, n) for n in names] == [getattr(c, n).data_ptr() for n in names]
    for n in names:
        setattr(c, n, getattr(c, n).clone())
        assert getattr(struct(c), n) == getattr(c, n).data_ptr()
    c.v_unit = c.v_unit.half()
    with pytest.raises(ValueError, match="units"):
        struct(c)
    with pytest.raises(ValueError, match="keys"):
        c.k = torch.zeros(3, 2, 4, 64, dtype=torch.uint8)


# ---------------------------------------------------------------- the references

@pytest.mark.parametrize("dim", [64, 128, 256])
def test_reference_layout_is_one_to_one(dim):
    at = kv4_ref.places(dim)
    assert sorted(at[0].ravel()) == list(range(64 * dim)) == sorted(at[2].ravel())
    for i in (1, 3):
        assert sorted(at[i][:, ::16].ravel()) == list(range(4 * dim))
        assert (at[i].reshape(64, -1, 16) == at[i][:, ::16, None]).all()
    rng = np.random.default_rng(dim)
    codes = rng.integers(0, 16, (2, 3, 64, dim)).astype(np.uint8)
    scales = rng.integers(0, 256, (2, 3, 64, dim // 16)).astype(np.uint8)
    for kind in "kv":
        a, b = kv4_ref.unpack(*kv4_ref.pack(codes, scales, kind), dim, kind)
        assert np.array_equal(a, codes) and np.array_equal(b, scales)


def test_reference_quantiser():
    # one group by hand: largest 12 with unit 0.5: 12 / 3 = 4 is a scale; a step of 2
    x = np.array([12.0, 0.5, 0.51, -1.5, 1.4, 2.5, 3.5, -5.0, 5.1, 7.0, 10.0, 10.1, 0, -0.0, 2, 8]).reshape(1, 1, 16)
    codes, scales = kv4_ref.quantise(x, [0.5])
    assert kv_ref.VALUES[scales].item() == 4.0
    assert kv4_ref.E2M1[codes].ravel().tolist() == [6, 0, .5, -1, .5, 1, 2, -2, 3, 4, 4, 6, 0, 0, 1, 4]
    assert kv4_ref.quantise(x * 1e6, [0.5])[1].item() == 0x7E                       # saturates
    assert kv4_ref.quantise(x * 1e-6, [0.5])[1].item() == 0                         # zeros
    assert kv4_ref.quantise(x * np.inf, [0.5])[1].item() == 0x7F


def test_reference_logprobs():
    z = np.log(np.array([[1, 2, 4, 1, 8]])).astype(np.float16)
    lp, h, ids, lps = kv4_ref.logprobs(z, [2], 4, 1.0)
    p = np.array([1, 2, 4, 1, 8]) / 16
    assert abs(lp[0] - math.log(0.25)) < 1e-3 and abs(h[0] + (p * np.log(p)).sum()) < 1e-3
    assert ids.tolist() == [[4, 2, 1, 0]] and abs(lps[0, 0] - math.log(0.5)) < 1e-3
