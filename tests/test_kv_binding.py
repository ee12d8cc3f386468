"""The binding of the speculative-round operators without a GPU: what it keeps between calls.  No kernel
is launched by any test here."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def kv():
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def host_tensors_pass(kv, monkeypatch):
    """The binding's check of a tensor without its place: pointers of host tensors are never followed here."""
    def need(t, dtype, dim, what):
        if t.dtype is dtype and t.dim() == dim and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(what)
    monkeypatch.setattr(kv, "_need", need)


def struct_of(kv, cache):
    """The struct that the next call gets."""
    ref = cache._checked() if hasattr(cache, "_checked") else cache._ref
    return ctypes.cast(ref, ctypes.POINTER(kv._Cache)).contents


def test_cache_follows_its_fields(kv, monkeypatch):
    # a cache that grows: calls go to the new tensors, whatever happens to the old ones
    host_tensors_pass(kv, monkeypatch)
    new = lambda pages, heads=2, dim=64: kv.KvCache.empty(pages, heads, dim, device="cpu")  # noqa: E731
    c, grown = new(3), new(5)
    assert struct_of(kv, c).pages == 3
    c.k = grown.k
    assert c.pages == 5
    with pytest.raises(ValueError, match="values"):       # four fields that do not agree yet
        struct_of(kv, c)
    c.v, c.k_scale = grown.v, grown.k_scale
    with pytest.raises(ValueError, match="scales"):
        struct_of(kv, c)
    c.v_scale = grown.v_scale
    s = struct_of(kv, c)
    assert (s.k, s.v, s.k_scale, s.v_scale) == tuple(t.data_ptr() for t in (c.k, c.v, c.k_scale, c.v_scale))
    assert (s.pages, s.heads, s.dim) == (c.pages, c.heads, c.dim) == (5, 2, 64)
    for name in ("k", "v", "k_scale", "v_scale"):          # one alone, of the same shape
        t = getattr(c, name).clone()
        setattr(c, name, t)
        assert getattr(struct_of(kv, c), name) == t.data_ptr()
    c.v = c.v.float()
    with pytest.raises(ValueError, match="values"):
        struct_of(kv, c)
    with pytest.raises(ValueError, match="keys"):
        c.k = torch.zeros(3, 2, 4, 64)
    wide = new(4, 3, 256)
    c.k, c.v, c.k_scale, c.v_scale = wide.k, wide.v, wide.k_scale, wide.v_scale
    s = struct_of(kv, c)
    assert (s.pages, s.heads, s.dim) == (c.pages, c.heads, c.dim) == (4, 3, 256)


def test_capture_is_asked_of_the_runtime(kv):
    assert kv.lib.hipStreamGetCaptureInfo            # (of the HIP runtime that the library is linked with)
