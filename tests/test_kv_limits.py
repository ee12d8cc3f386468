"""The speculative-round operators without a GPU: bounds of products of sizes, sizes of scratch, and
what the binding checks and keeps.  No kernel is launched by any test here."""
import ctypes

import pytest
import torch

P = 1 << 20          # a well-aligned address; argument checks never follow it
NULL, SHAPE, DEVICE = 1, 2, 5


@pytest.fixture(scope="module")
def kv():
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def cache(kv, heads, dim=64, pages=10):
    return ctypes.byref(kv._Cache(P, P, P, P, pages, heads, dim))


@pytest.mark.parametrize("rows,q_heads,heads,ok", [(1 << 20, 1024, 1024, True), (1 << 20, 2048, 1024, False),
                                                   (1 << 14, 65536, 1024, True), ((1 << 14) + 1, 65536, 1024, False)])
def test_attention_bounds_rows_times_heads(kv, rows, q_heads, heads, ok):
    if ok and torch.cuda.is_available():
        pytest.skip("a GPU is present: a call that passes its checks would be launched")
    s = q_heads * 64
    got = kv.lib.qpn_kv_attention(cache(kv, heads), P, s, P, s, q_heads, rows, 1, rows, P, P, P, 8, 8, 0.1, 0, P, 0, None)
    assert got == (DEVICE if ok else SHAPE)


def test_append_bounds_rows_times_heads(kv):
    s = 2048 * 64
    call = lambda rows: kv.lib.qpn_kv_rope_append(  # noqa: E731
        cache(kv, 512), P, s, rows, 1024, None, None, 1e-6, P, 64, 0, P, P, P, 1024 * 64, None)
    assert call((1 << 30) // 1536 + 1) == SHAPE
    assert call((1 << 25) // 512 + 1) == SHAPE
    if not torch.cuda.is_available():
        assert call((1 << 25) // 512) == DEVICE
    assert call(0) == 0


def test_scratch_grows_with_what_it_holds(kv):
    a = kv.attention_scratch_bytes
    assert a(1, 8, 40, 8, 128, 8) == kv.SCRATCH_ZEROED and a(1, 8, 40, 8, 128, 9) > kv.SCRATCH_ZEROED
    assert a(4096, 64, 40, 8, 128, 1000) == kv.SCRATCH_ZEROED        # more segments than pieces: nothing is cut
    assert a(0, 0, 40, 8, 128, 0) == kv.SCRATCH_ZEROED
    assert a(1, 8, 8, 1, 256, 4096) < 1 << 32
    v = kv.verify_scratch_bytes
    assert v(0, 0, 1) >= kv.SCRATCH_ZEROED
    assert v(8, 1, 4096) < v(8, 1, 1 << 20) < v(9, 1, 1 << 20) < v(9, 2, 1 << 20)
    assert v(65535, 4096, 1) < 1 << 40


def test_round_is_checked_again_when_a_field_is_set(kv):
    e = lambda n: torch.empty(n, dtype=torch.int32)  # noqa: E731
    r = kv.Round(e(3), e(4), e(3), e(1), e(9), e(9))
    with pytest.raises(ValueError):           # host tensors
        r._checked()
    r.__dict__["_args"] = "checked"
    r.slots = e(8)
    assert r._args is None                    # what was checked belonged to the old field
    with pytest.raises(ValueError, match="do not agree"):
        r._checked()
    for name, size in (("row_start", 3), ("held", 2), ("free_count", 2), ("positions", 8)):
        r = kv.Round(e(3), e(4), e(3), e(1), e(9), e(9))
        setattr(r, name, e(size))
        with pytest.raises(ValueError, match="do not agree"):
            r._checked()


def test_binding_refuses_sizes_that_disagree(kv):
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    h = lambda *n: torch.zeros(*n, dtype=torch.float16)  # noqa: E731

    class Stand:                               # (what the checks read of a cache)
        dim, heads = 64, 2
    with pytest.raises(ValueError):
        kv.plan_round(i(2), i(2), i(2), i(2, 3), i(4), i(1))                    # neither capacity nor out
    with pytest.raises(ValueError):
        kv.attention(Stand, h(3, 100), i(2), i(1), i(1, 3), 3)                  # no whole heads
    with pytest.raises(ValueError):
        kv.attention(Stand, h(3, 128), i(3), i(1), i(1, 3), 3)                  # row_start of another length
    with pytest.raises(ValueError):
        kv.rope_append(Stand, h(3, 512), 4, i(2), i(3), None)                   # host rows, and positions too short
    with pytest.raises(ValueError):
        kv.verify_sampled(h(3, 9), i(3), i(2), torch.zeros(3), torch.zeros(1))  # host logits
