"""The speculative-round operators at the edges of what they accept.

References and tolerances are those of test_gpu_kv.py; where one differs it is derived at its test.
"""
import threading
import time

import numpy as np
import pytest
import torch

import kv_ref
from gpu_util import dev, host, need_gpu
from test_gpu_kv import PAGE, AttnCase, append_case, i32, run_slots, verify_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    need_gpu()
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


# ---------------------------------------------------------------- attention

# few and many rows of a KV head; the second request is the one longer than its table
@pytest.mark.parametrize("dim,hq,hk", [(64, 4, 2), (128, 2, 2), (256, 8, 1)])
@pytest.mark.parametrize("rows,tokens", [(8, 6), (100, 90), (200, 256), (200, 300)])
def test_attention_more_rows_than_the_table_has_places(kv, dim, hq, hk, rows, tokens):
    # the table holds fewer tokens than the request has rows: all of its rows are NaN, those that
    # would stand before the first token of the table too
    width = -(-tokens // PAGE) - 1                 # 0 pages for 6 tokens, 1 for 90, 3 and 4
    c = AttnCase(kv, [(2, PAGE * max(width, 1)), (rows, tokens), (1, 5)], hq, hk, dim, 50)
    c.table = c.table[:, :width]
    if width == 0:
        c.seq = [0, tokens, -3]
    y = c.run()
    assert np.isnan(y[2:2 + rows]).all()
    if width == 0:
        assert not y[:2].any() and not y[2 + rows:].any()
    else:
        assert np.isfinite(y[:2]).all() and np.isfinite(y[2 + rows:]).all()
    # alone, the call's work is cut in another way
    c.q, c.row_start, c.seq, c.table, c.lens = c.q[2:2 + rows], np.array([0, rows]), [tokens], c.table[1:2], c.lens[1:2]
    assert np.isnan(c.run()).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(5, 3), (4, 0), (2, 100), (3, 1)], [(70, 3), (60, 0), (50, 100), (90, 70)], [(8, 3)],
                                  [(300, 200)]])
def test_attention_windows_of_rows_before_the_first_token(kv, dim, lens):
    # fewer tokens than rows, and windows up to the widest: from the tokens' number on a window hides nothing
    c = AttnCase(kv, lens, 4, 2, dim, 54)
    clean = c.run()
    c.check(clean)
    c.check(c.run(window=1), 1)
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 200, 2 ** 30):
        assert np.array_equal(c.run(window=window), clean), window


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,tokens", [(8, 130), (70, 150)])
@pytest.mark.parametrize("scale", [np.nan, np.inf, -np.inf, -2.0])
def test_attention_bad_value_scale_reaches_only_rows_that_see_the_page(kv, dim, rows, tokens, scale):
    c = AttnCase(kv, [(rows, tokens), (rows, 64)], 4, 2, dim, 55)
    first, heads = tokens - rows, slice(2, 4)      # the first row's position; the query heads of KV head 1
    good = c.scale.copy()
    for window, page in ((0, 2), (3, 1), (0, 1)):
        clean = c.run(window=window)
        c.scale[1, c.table[0, page], 1] = scale
        y = c.run(window=window)
        c.scale = good.copy()
        hit = np.zeros(y.shape, bool)
        for i in range(rows):
            low = max(0, first + i + 1 - window) if window else 0
            hit[i, heads] = first + i >= PAGE * page and low < PAGE * (page + 1)
        assert hit.any() and np.array_equal(np.isnan(y), hit), (window, page)
        c.check(np.where(hit, clean, y), window)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,hq", [(2, 2), (64, 2), (60, 1)])
@pytest.mark.parametrize("tokens", [64 * 6, 64 * 40])
@pytest.mark.parametrize("ratio", [4, 8, 13, 16, 19, 24])
def test_attention_weights_on_a_page_of_small_scale(kv, dim, rows, hq, tokens, ratio):
    # All weight lies on page 3, whose values have a scale 2^ratio below the others'.  An output then is
    # as exact as with equal scales: FP16 weights are off by 2^-11 of each, or 2^-25 of the row's largest
    # below 2^-14 of it (and by no more than a weight itself), whatever the scales of other pages.
    c = AttnCase(kv, [(rows, tokens)], hq, 1, dim, 56 + ratio)
    page = c.table[0, 3]
    c.codes[0] = 0xB8                              # keys: -1
    c.codes[0, page] = 0x38                        # and 1 on the page, but for the first dimension: -1 .. 1
    c.codes[0, page, :, :, 0] = np.random.default_rng(57).integers(0, 0x39, PAGE) | (np.arange(PAGE) % 2 * 0x80)
    c.scale[0] = 1.0
    c.scale[1] = 2.0 ** 10
    c.scale[1, page] = 2.0 ** (10 - ratio)
    c.q[:] = 20 / dim ** 0.5                       # scores +-20 by the page, +-6 within it
    c.q[:, :, 0] = 6 * dim ** 0.5
    y = c.run()
    k, v = c.values()
    ref, mag = kv_ref.attention(c.q.astype(np.float64), k, v, c.row_start, c.seq, np.clip(c.table, 0, None), dim ** -0.5, 0)
    ids = c.table[0, :tokens // PAGE]
    kk, vv = k[ids, 0].reshape(-1, dim), np.abs(v[ids, 0].reshape(-1, dim))
    s = kk @ c.q[0, 0].astype(np.float64) * dim ** -0.5          # (all rows ask the same)
    assert np.ptp(s) > 35 and s.argmax() // PAGE == 3
    small = np.minimum(2.0 ** -25, np.exp(s - s.max())) @ vv
    tol = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -24 * (40 * dim + tokens)) * mag + small + 2.0 ** -25
    err = np.abs(y - ref)
    assert (err <= tol).all(), f"max error {(err / tol).max():.2f} of what is allowed, {(err > tol).sum()} outside"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [4, 64])
def test_attention_value_scales_over_the_whole_range(kv, dim, rows):
    # page scales from what a page of zeros has to what FP16 cannot hold any more, in rising, falling and mixed order
    c = AttnCase(kv, [(rows, 64 * 9 + 5)], 2, 1, dim, 58)
    for powers in (np.linspace(-60, 9, 10), np.linspace(9, -60, 10), np.array([-60, 9, -30, 0, 9, -60, 4, -20, 1, -45])):
        c.scale[1][c.table[0, :10], 0] = 2.0 ** np.round(powers)
        c.check(c.run())
    c.scale[1][c.table[0, :10], 0] = 2.0 ** np.array([-60, 100, -60, 0, 100, -100, 4, -149, 1, -45])
    y = c.run()
    ref, mag = kv_ref.attention(c.q.astype(np.float64), *c.values(), c.row_start, c.seq, np.clip(c.table, 0, None), dim ** -0.5, 0)
    far = np.abs(ref) > 1e6 + 2.0 ** -10 * mag     # beyond FP16, and of a sign that rounded weights cannot change
    assert far.mean() > 0.9 and (mag > 1e20).all() and np.isinf(y).all()
    wrong = far & (y != np.copysign(np.inf, ref))
    assert not wrong.any(), f"{wrong.sum()} signs, up to {(np.abs(ref) / mag)[wrong].max():.2e} of the magnitude"


# ---------------------------------------------------------------- rope_append

def halfway_values(scale):
    """The FP16 values x > 0 with x / scale halfway between two E4M3 values (exactly, in 64 bits)."""
    x = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    x = x[x <= 224]                                # (larger ones would raise a scale between 1/2 and 1)
    return x[np.isin(x / scale, (kv_ref.VALUES[1:127] + kv_ref.VALUES[:126]) / 2)]


@pytest.mark.parametrize("scale", [0.8046875, 0.8359375, 0.9140625, 0.9609375, 0.92578125])
def test_append_ties_of_scales_that_are_no_power_of_two(kv, scale):
    # a page keeps its former scale s, of any 24 bits; a value halfway between two codes goes to the
    # even one, which x * (1 / s) misses where that product is rounded off the middle
    ties = halfway_values(scale)
    off = kv_ref.e4m3_codes(ties / scale) != kv_ref.e4m3_codes(ties * (1.0 / scale))
    assert off.any()
    rows, hq, hk, dim = 3, 2, 1, 64
    x = np.resize(ties, (rows, (hq + 2 * hk) * dim)) * np.where(np.arange(rows) % 2, -1.0, 1.0)[:, None]
    x[2, (hq + hk) * dim] = np.inf                 # saturates
    x[2, (hq + hk) * dim + 1] = np.nan
    append_case(kv, dim, hq, hk, [5, 6, 17], [5, 6, 17], 1, 51, rot=0, norm=False, x=x.astype(np.float16), old=scale)


def test_append_odd_scales_of_rotated_keys(kv):
    slots, pos = run_slots([(1000, 300), (70, 30), (63, 66)], 14, 52)
    for old in (0.0123, 0.7, 37.3):
        append_case(kv, 128, 4, 2, slots, pos, 14, 53, old=old)


# ---------------------------------------------------------------- scratch

class Watched:
    """Stands before the library: notes the scratch of each call, and calls that have one at the same time."""

    def __init__(self, lib, launch):
        self.lib, self.launch, self.given, self.inside, self.clashes = lib, launch, [], [], 0

    def __getattr__(self, name):
        f = getattr(self.lib, name)
        if name not in ("qpn_kv_attention", "qpn_kv_verify_sampled"):
            return f

        def call(*args):
            scratch = args[-3]                     # .., scratch, its bytes, stream
            self.given.append(scratch)
            if self.launch:
                return f(*args)
            self.clashes += scratch in self.inside
            self.inside.append(scratch)
            time.sleep(0.002)                      # (another thread may run)
            self.inside.remove(scratch)
            return 0
        return call


def attention_call(kv, seed=60, tokens=3000):
    """A call whose pieces meet in the scratch: (call(stream, out), its outputs' bits)."""
    c = AttnCase(kv, [(8, tokens)], 10, 2, 128, seed)
    q, row_start, seq, table, cache = dev(c.q.reshape(8, -1)), i32(c.row_start), i32(c.seq), i32(c.table), c.device()
    return (lambda stream=None, out=None: kv.attention(cache, q, row_start, seq, table, 8, stream=stream, out=out),
            c.run().reshape(8, -1))


def test_threads_do_not_share_a_scratch_at_the_same_time(kv, monkeypatch):
    # a call of two launches hands its sums over through the scratch: on one stream, the launches of two
    # threads' calls must not come in turn
    call, _ = attention_call(kv)
    _, _, args = verify_case(kv, [4, 4], 5000, 61, True)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream), kv.verify_sampled(*args, stream=stream)
    torch.cuda.synchronize()
    watch = Watched(kv.lib, launch=False)
    monkeypatch.setattr(kv, "lib", watch)
    failed = []

    def work(f):
        try:
            for _ in range(10):
                f()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(f,)) for f in (
        lambda: call(stream), lambda: kv.verify_sampled(*args, stream=stream), lambda: call(stream))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(watch.given) == 30 and watch.clashes == 0


def test_graphs_of_a_stream_have_scratch_of_their_own(kv, monkeypatch):
    # the stream has a scratch already; graphs captured on it may run beside each other and beside its calls
    calls = [attention_call(kv, 62), attention_call(kv, 63, 6000)]
    stream, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for call, want in calls:
        assert np.array_equal(host(call(stream)), want)
    watch = Watched(kv.lib, launch=True)
    monkeypatch.setattr(kv, "lib", watch)
    held = {s.data_ptr() for s in kv._scratches.values()}
    graphs, outs = [], []
    for call, want in calls:
        g, out = torch.cuda.CUDAGraph(), [torch.zeros(want.shape, dtype=torch.float16, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        before = len(watch.given)
        with torch.cuda.graph(g, stream=stream):
            for o in out:
                call(out=o)
        mine = set(watch.given[before:])
        assert len(mine) == 1 and not mine & held  # one for the graph's calls, and nobody else's
        held |= mine
        graphs.append(g)
        outs.append(out)
    for _ in range(4):
        for out in outs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, others):
            with torch.cuda.stream(s):
                g.replay()
        eager = [calls[0][0](stream) for _ in range(3)]
        torch.cuda.synchronize()
        for o in eager:
            assert np.array_equal(host(o), calls[0][1])
        for out, (_, want) in zip(outs, calls):
            for o in out:
                assert np.array_equal(host(o), want)


def test_scratch_that_grows_within_a_capture(kv):
    calls = [attention_call(kv, 64, 700), attention_call(kv, 65, 6000)]
    stream, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    outs = [torch.zeros(8, 1280, dtype=torch.float16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        for i, o in enumerate(outs):
            calls[i % 2][0](out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert np.array_equal(host(o), calls[i % 2][1])
        assert np.array_equal(host(calls[0][0]()), calls[0][1])


def test_scratch_that_is_given_is_checked(kv):
    c = AttnCase(kv, [(2, 100)], 4, 2, 64, 66)
    args = (c.device(), dev(c.q.reshape(2, -1)), i32(c.row_start), i32(c.seq), i32(c.table), 2)
    _, _, verify = verify_case(kv, [2], 100, 67, False)
    size = kv.SCRATCH_ZEROED + (1 << 20)
    for bad in (torch.zeros(size, dtype=torch.uint8),                                   # on the host
                torch.zeros(size, dtype=torch.float32, device="cuda"),
                torch.zeros(2, size, dtype=torch.uint8, device="cuda"),
                torch.zeros(2 * size, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="scratch"):
            kv.attention(*args, scratch_=bad)
        with pytest.raises(ValueError, match="scratch"):
            kv.verify_sampled(*verify, scratch_=bad)
    s = torch.zeros(size, dtype=torch.uint8, device="cuda")
    assert np.array_equal(host(kv.attention(*args, scratch_=s)).reshape(c.q.shape), c.run())
    assert int(s[:kv.SCRATCH_ZEROED].count_nonzero()) == 0
