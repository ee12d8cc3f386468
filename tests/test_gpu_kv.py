"""GPU parity of the speculative-round operators against plain FP64 references (kv_ref.py).

Tolerances, derived before the first run:
  queries of rope_append   FP16 rounding 2^-11 |y|, FP32 arithmetic and the hardware sine and cosine
                           (2^-18 of the pair's length), FP16 subnormals 2^-25;
  codes and scales         equal (keys are computed in 64 bits; the seeds are fixed);
  attention                2^-11 |y| (output) + 2^-11 a (each weight rounded to FP16) +
                           2^-24 (dim s + tokens) a (FP32 scores up to s = 40 and sums), a = sum w |v| / sum w,
                           + tokens 2^-25 max |v| (weights below FP16's normal range, the largest being
                           at least 1) + 2^-25;
  verification             tokens and counts equal; probabilities 2^-23 |p| + 1e-10.
"""
import numpy as np
import pytest
import torch

import kv_ref
from gpu_util import dev, host, log, need_gpu

pytestmark = pytest.mark.gpu
PAGE = kv_ref.PAGE


@pytest.fixture(scope="module")
def kv():
    need_gpu()
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f8(codes):
    return dev(codes).view(torch.float8_e4m3fn)


def bytes_of(t):
    return host(t.view(torch.uint8))


# ---------------------------------------------------------------- plan_round

def check_plan(kv, before, rows, held, table, free, count, capacity, out=None, alias=False):
    ref = kv_ref.plan_round(before, rows, held, table, free, count, capacity)
    td, fc, hd = i32(table), i32([count]), i32(held)
    if alias:
        out = kv.Round.empty(len(before), capacity)
        out.held, out.free_count = hd, fc
    r = kv.plan_round(i32(before), i32(rows), hd, td, i32(free), fc, None if alias else capacity, out=out)
    for name in ("seq_lens", "row_start", "held", "free_count", "slots", "positions"):
        assert host(getattr(r, name)).tolist() == list(ref[name]), name
    assert np.array_equal(host(td), ref["table"])


@pytest.mark.parametrize("n,most,tokens,seed", [(1, 1, 0, 0), (1, 8, 60, 1), (1, 256, 1000, 2), (3, 8, 64, 3), (64, 8, 900, 4),
                                                (257, 5, 300, 5), (1025, 3, 130, 6), (4096, 2, 70, 7), (5, 700, 10, 8)])
def test_plan_round(kv, n, most, tokens, seed):
    rng = np.random.default_rng(seed)
    before = rng.integers(0, tokens + 1, n)
    rows = rng.integers(0, most + 1, n)
    held = -(-before // PAGE) + rng.integers(0, 2, n)
    width = int(-(-(before + rows).max() // PAGE)) + 2
    table = rng.integers(0, 5000, (n, width))
    need = np.maximum(0, -(-(before + rows) // PAGE) - held).sum()
    free = rng.permutation(int(need) + 9)
    for count in (need + 9, need, max(need - 1, 0), need // 2, 0, -3):
        for capacity in (int(rows.sum()) + 5, max(int(rows.sum()) // 2, 1)):
            check_plan(kv, before, rows, held, table, free, int(count), capacity)
    check_plan(kv, before, rows, held, table, free, int(need) + 99, int(rows.sum()) + 1, alias=True)


def test_plan_round_malformed_requests(kv):
    # negative lengths, more pages held than the table is wide, tokens without pages, past the table
    before, rows = [5, -1, 3, 100, 10, 700, 64], [2, 1, -2, 1, 1, 1, 1]
    held = [1, 0, 1, 1, 99, 11, 1]
    check_plan(kv, before, rows, held, np.zeros((7, 8), int), np.arange(20, 30), 10, 12)


def test_plan_round_empty(kv):
    check_plan(kv, [], [], [], np.zeros((0, 4), int), np.arange(3), 3, 4)
    check_plan(kv, [0, 0], [0, 0], [0, 0], np.zeros((2, 0), int), np.zeros(0, int), 0, 0)


# ---------------------------------------------------------------- rope_append

def append_case(kv, dim, hq, hk, slots, positions, pages, seed, rot=None, interleaved=False, norm=True, x=None,
                stride=0, inplace=False, old=None, stream=None):
    rng = np.random.default_rng(seed)
    rows, rot = len(slots), dim if rot is None else rot
    if x is None:
        x = (rng.standard_normal((rows, (hq + 2 * hk) * dim)) * 10.0 ** rng.uniform(-1, 1, (rows, 1))).astype(np.float16)
    qw, kw = ((1 + 0.3 * rng.standard_normal((2, dim))).astype(np.float16) if norm else (None, None))
    f = (1e6 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    codes = rng.integers(0, 256, (2, pages, hk, PAGE, dim)).astype(np.uint8)
    codes[codes % 128 == 127] = 3
    scale = 2.0 ** rng.integers(-12, -3, (2, pages, hk)).astype(np.float32) if old is None else np.full((2, pages, hk), old, np.float32)
    cache = kv.KvCache(f8(kv_ref.pack_k(codes[0])), f8(kv_ref.pack_v(codes[1])), dev(scale[0]), dev(scale[1]))
    xd = torch.zeros(rows, x.shape[1] + stride, dtype=torch.float16, device="cuda")
    xd[:, :x.shape[1]] = dev(x)
    xd = xd[:, :x.shape[1]]
    out = xd[:, :hq * dim] if inplace else None
    log(f"append dim {dim} heads {hq}/{hk} rows {rows} rot {rot} seed {seed}")
    torch.cuda.synchronize()
    q = kv.rope_append(cache, xd, hq, i32(positions), i32(slots), dev(f) if rot else None,
                       None if qw is None else dev(qw), None if kw is None else dev(kw), 1e-6, interleaved, out=out,
                       stream=stream)
    torch.cuda.synchronize()
    xs = x.astype(np.float64).reshape(rows, hq + 2 * hk, dim)
    with np.errstate(invalid="ignore"):
        q_ref = kv_ref.norm_rope(xs[:, :hq], qw, 1e-6, f, interleaved, positions).reshape(rows, -1)
        k_ref = kv_ref.norm_rope(xs[:, hq:hq + hk], kw, 1e-6, f, interleaved, positions)
        want, ws = codes.copy(), scale.astype(np.float64)
        kv_ref.append(want[0], ws[0], k_ref, slots)
        kv_ref.append(want[1], ws[1], xs[:, hq + hk:], slots)
    got = host(q).astype(np.float64)
    length = np.abs(q_ref).reshape(rows, hq, dim).max(-1).repeat(dim, 1).reshape(rows, -1)
    ok = np.isfinite(q_ref)
    assert np.array_equal(np.isnan(got), np.isnan(q_ref))
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - q_ref) <= 2.0 ** -11 * np.abs(q_ref) + 2.0 ** -17 * length + 2.0 ** -25)[ok].all()
    assert np.array_equal(host(cache.k_scale), ws[0]) and np.array_equal(host(cache.v_scale), ws[1])
    gk, gv = kv_ref.unpack_k(bytes_of(cache.k)), kv_ref.unpack_v(bytes_of(cache.v))
    # NaN has two codes; the sign of one is not specified
    same = lambda a, b: np.array_equal(np.where(a % 128 == 127, 127, a), np.where(b % 128 == 127, 127, b))  # noqa: E731
    assert same(gk, want[0]), f"{(gk != want[0]).sum()} key codes differ"
    assert same(gv, want[1]), f"{(gv != want[1]).sum()} value codes differ"


def run_slots(starts, pages, seed):
    """Slots and positions of requests with (tokens before, rows) on distinct pages."""
    ids = list(np.random.default_rng(seed).permutation(pages))
    slots, pos = [], []
    for before, rows in starts:
        page = {}
        for t in range(before, before + rows):
            slots.append(page.setdefault(t // PAGE, ids[0] if t // PAGE not in page else 0) * PAGE + t % PAGE)
            if page[t // PAGE] == ids[0]:
                ids.pop(0)
            pos.append(t)
    return slots, pos


@pytest.mark.parametrize("dim,hq,hk", [(128, 40, 8), (64, 4, 4), (256, 8, 1), (128, 10, 2), (64, 64, 1)])
@pytest.mark.parametrize("starts", [[(0, 1)], [(1777, 1)], [(4090, 8)], [(63, 2), (0, 7)], [(100, 150)], [(64, 64), (5, 3)]])
def test_append(kv, dim, hq, hk, starts):
    slots, pos = run_slots(starts, 12, dim)
    append_case(kv, dim, hq, hk, slots, pos, 12, dim + len(slots))


@pytest.mark.parametrize("rot,interleaved,norm", [(128, True, True), (64, False, True), (32, True, False), (0, False, True),
                                                  (0, False, False), (112, False, False), (16, False, True)])
def test_append_rotations(kv, rot, interleaved, norm):
    slots, pos = run_slots([(130001, 9), (70, 20)], 6, 1)
    append_case(kv, 128, 6, 2, slots, pos, 6, rot + norm, rot=rot, interleaved=interleaved, norm=norm)


def test_append_many_requests(kv):
    # more than one step of heads per wavefront, a page for each request
    slots, pos = run_slots([(37 * i % 500, 1 + i % 4) for i in range(200)], 420, 2)
    append_case(kv, 128, 40, 8, slots, pos, 420, 3)


def test_append_slots_in_any_order(kv):
    # rows of one page scattered over the call, one slot twice, padding, slots out of range
    rng = np.random.default_rng(5)
    slots = list(rng.permutation(3 * PAGE)[:70]) + [-1, 7, 7, -5, 4 * PAGE, 2 ** 31 - 1, 7]
    append_case(kv, 64, 4, 2, slots, rng.integers(0, 900, len(slots)), 4, 6)


@pytest.mark.parametrize("old", [2.0 ** -20, 2.0 ** -9, 2.0 ** 3, 0.0123])
def test_append_growing_scale(kv, old):
    # far below the new values (codes round to few steps or zero), near, above, and no power of two
    slots, pos = run_slots([(60, 3), (33, 1), (50, 30)], 6, 3)
    append_case(kv, 128, 4, 2, slots, pos, 6, 8, old=old)


def test_append_special_values(kv):
    rows, hq, hk, dim = 6, 4, 2, 64
    x = np.random.default_rng(9).standard_normal((rows, (hq + 2 * hk) * dim)).astype(np.float16)
    x[1, :] = 0.0                          # a row of zeros
    x[2, (hq + hk) * dim + 3] = np.inf     # an infinite value saturates, and does not set the scale
    x[3, (hq + hk) * dim + 4] = np.nan     # NaN codes stay with their element
    x[4, hq * dim + 5] = np.nan            # a NaN key makes its whole head NaN
    x[5, :] = 6e-8                         # FP16 subnormals
    append_case(kv, dim, hq, hk, [0, 1, 2, 3, 4, 5], [9, 8, 7, 6, 5, 4], 2, 10, x=x)
    append_case(kv, dim, hq, hk, [70, 71, 72, 73, 74, 75], [9, 8, 7, 6, 5, 4], 2, 10, x=x, norm=False)
    append_case(kv, dim, hq, hk, [0] + [-1] * 5, [0] * 6, 1, 11, x=np.zeros_like(x))


def test_append_strides_in_place_and_streams(kv):
    slots, pos = run_slots([(4090, 8)], 4, 4)
    append_case(kv, 128, 10, 2, slots, pos, 4, 12, stride=24)
    append_case(kv, 128, 10, 2, slots, pos, 4, 13, inplace=True)
    append_case(kv, 128, 10, 2, slots, pos, 4, 14, stream=torch.cuda.Stream())


# ---------------------------------------------------------------- attention

class AttnCase:
    """lens: (rows, tokens in all) of each request."""

    def __init__(self, kv, lens, hq, hk, dim, seed, extra_pages=2, size=2.0):
        rng = np.random.default_rng(seed)
        self.kv, self.lens, self.hq, self.hk, self.dim = kv, lens, hq, hk, dim
        need = [max(0, -(-t // PAGE)) for _, t in lens]
        pages = sum(need) + extra_pages
        self.codes = rng.integers(0, 256, (2, pages, hk, PAGE, dim)).astype(np.uint8)
        self.codes &= 0xBF                       # |value| < 2: scales below make them of unit size
        self.scale = 2.0 ** rng.integers(-2, 3, (2, pages, hk)).astype(np.float32)
        ids = rng.permutation(pages)
        self.width = max(need) + 1
        self.table = np.full((len(lens), self.width), -7, np.int64)   # entries past the length are junk
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n]
            at += n
        self.row_start = np.concatenate([[0], np.cumsum([r for r, _ in lens])]).astype(int)
        self.q = (size * rng.standard_normal((max(1, self.row_start[-1]), hq, dim)) / dim ** 0.25).astype(np.float16)
        self.seq = [t for _, t in lens]

    def values(self):
        v = kv_ref.VALUES[self.codes] * self.scale[..., None, None]
        return v[0], v[1]

    def device(self):
        return self.kv.KvCache(f8(kv_ref.pack_k(self.codes[0])), f8(kv_ref.pack_v(self.codes[1])), dev(self.scale[0]),
                               dev(self.scale[1]))

    def run(self, cache=None, window=0, **more):
        q = dev(self.q.reshape(self.q.shape[0], -1))
        cache = self.device() if cache is None else cache
        log(f"attention {self.lens[:4]}.. heads {self.hq}/{self.hk} dim {self.dim} window {window}")
        torch.cuda.synchronize()
        y = self.kv.attention(cache, q, i32(self.row_start), i32(self.seq), i32(self.table), max(r for r, _ in self.lens),
                              window=window, **more)
        return host(y).reshape(self.q.shape).astype(np.float64)

    def check(self, y, window=0, rows=None):
        k, v = self.values()
        table = np.clip(self.table, 0, None)
        ref, mag = kv_ref.attention(self.q.astype(np.float64), k, v, self.row_start, self.seq, table, self.dim ** -0.5, window)
        tokens = max(max(self.seq), 1)
        vmax = np.nanmax(np.abs(v))
        tol = (2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -24 * (40 * self.dim + tokens)) * mag
               + tokens * 2.0 ** -25 * vmax + 2.0 ** -25)
        rows = slice(None) if rows is None else rows
        err = np.abs(y - ref)[rows]
        assert np.isfinite(y[rows]).all()
        assert (err <= tol[rows]).all(), f"max error {err.max():.3e}, {(err > tol[rows]).sum()} outside"
        return ref


@pytest.mark.parametrize("dim,hq,hk", [(128, 40, 8), (128, 5, 1), (64, 8, 8), (64, 16, 1), (256, 8, 2), (128, 6, 2)])
@pytest.mark.parametrize("rows,tokens", [(1, 1), (1, 63), (1, 64), (1, 65), (8, 8), (8, 200), (3, 1000), (8, 4099), (1, 3001)])
def test_attention(kv, dim, hq, hk, rows, tokens):
    c = AttnCase(kv, [(rows, tokens)], hq, hk, dim, dim + tokens)
    c.check(c.run())


@pytest.mark.parametrize("dim,hq,hk,rows,tokens", [(128, 40, 8, 256, 700), (64, 4, 1, 100, 1000), (256, 4, 2, 70, 300),
                                                   (128, 16, 2, 33, 64), (128, 8, 8, 64, 2048)])
def test_attention_prompt_blocks(kv, dim, hq, hk, rows, tokens):
    c = AttnCase(kv, [(rows, max(rows, tokens))], hq, hk, dim, rows)
    c.check(c.run())


RAGGED = [(8, 300), (1, 1), (0, 500), (3, 3), (8, 64), (5, 1300), (1, 129), (0, 0), (2, 4000), (7, 70)]


@pytest.mark.parametrize("dim,hq,hk", [(128, 10, 2), (64, 4, 4), (256, 16, 1)])
@pytest.mark.parametrize("window", [0, 1, 64, 100, 5000])
def test_attention_ragged_and_windows(kv, dim, hq, hk, window):
    c = AttnCase(kv, RAGGED, hq, hk, dim, 5)
    c.check(c.run(window=window), window)


def test_attention_many_requests(kv):
    lens = [(1 + i % 3, 3 + (i * 97) % 700) for i in range(300)]
    c = AttnCase(kv, lens, 4, 2, 64, 6)
    c.check(c.run())


@pytest.mark.parametrize("window", [0, 40])
def test_attention_unseen_tokens_never_matter(kv, window):
    # NaN and the largest codes in everything no row may see; NaN values in tokens that only later
    # rows see reach those rows alone
    c = AttnCase(kv, [(6, 150), (2, 64), (4, 321)], 10, 2, 128, 7)
    clean = c.run(window=window)
    used = np.zeros(c.codes.shape[1:4], bool)
    for r, (n, t) in enumerate(c.lens):
        for j in range(max(0, t - n + 1 - window) if window else 0, t):
            used[c.table[r, j // PAGE], :, j % PAGE] = True
    for junk in (0x7F, 0xFF, 0x7E):
        codes = c.codes.copy()
        c.codes[:, ~used] = junk
        assert np.array_equal(c.run(window=window), clean), hex(junk)
        c.codes = codes
    # request 0, KV head 1: the value of its row 3's own token (position 147), dimension 17
    p = 147
    c.codes[1, c.table[0, p // PAGE], 1, p % PAGE, 17] = 0x7F
    y = c.run(window=window)
    want = np.isnan(y)
    hit = np.zeros_like(want)
    hit[3:6, 5:10, 17] = True
    assert np.array_equal(want, hit)
    assert np.array_equal(y[~hit], clean[~hit])
    # and a NaN key makes the whole of those rows NaN
    c.codes[0, c.table[0, p // PAGE], 1, p % PAGE, 3] = 0xFF
    y = c.run(window=window)
    hit[3:6, 5:10, :] = True
    assert np.array_equal(np.isnan(y), hit)


def test_attention_rows_that_see_nothing(kv):
    # fewer tokens than rows: the first rows stand before the first token
    c = AttnCase(kv, [(5, 3), (4, 0), (2, 100), (3, 1)], 8, 2, 64, 8)
    y = c.run()
    c.check(y)
    assert not y[:2].any() and not y[5:9].any() and not y[11:13].any() and y[2:5].any(-1).all()
    c.seq = [-4, -2 ** 31, 100, 1]
    y = c.run()
    assert not y[:9].any() and y[9:11].any()


def test_attention_bad_pages_and_lengths(kv):
    c = AttnCase(kv, [(2, 200), (3, 200), (2, 90)], 8, 2, 64, 9)
    clean = c.run()
    for bad in (-1, c.codes.shape[1], 2 ** 31 - 1):
        keep = c.table.copy()
        c.table[1, 2] = bad
        y = c.run()
        assert np.isnan(y[2:5]).all()
        assert np.array_equal(y[[0, 1, 5, 6]], clean[[0, 1, 5, 6]])
        c.table = keep
    c.seq = [200, 64 * c.width + 1, 90]
    y = c.run()
    assert np.isnan(y[2:5]).all() and np.array_equal(y[[0, 1, 5, 6]], clean[[0, 1, 5, 6]])
    # requests whose rows are out of order or past the end are skipped
    c.seq = [200, 200, 90]
    c.row_start = np.array([0, 2, 1, 900])
    q = dev(c.q.reshape(7, -1))
    out = torch.full_like(q, 3.0)
    kv.attention(c.device(), q, i32(c.row_start), i32(c.seq), i32(c.table), 3, out=out)
    y = host(out).reshape(c.q.shape)
    assert np.array_equal(y[:2], clean[:2]) and (y[2:] == 3.0).all()


def test_attention_infinite_queries(kv):
    c = AttnCase(kv, [(3, 100)], 4, 1, 64, 10)
    clean = c.run()
    c.q[1, 2, 5] = np.inf
    c.q[2, 0, 0] = np.nan
    y = c.run()
    hit = np.zeros(y.shape, bool)
    hit[1, 2] = hit[2, 0] = True
    assert np.isnan(y[hit]).all() and np.array_equal(y[~hit], clean[~hit])


def test_attention_peaked_scores_and_scales(kv):
    # scores up to +-40 (one token takes all, wherever it lies) and page scales over 2^40
    c = AttnCase(kv, [(8, 1500)], 10, 2, 128, 11, size=8.0)
    c.scale[1] *= 2.0 ** np.random.default_rng(0).integers(-20, 1, c.scale[1].shape)
    c.check(c.run())
    c.scale[1] = 0.0
    assert not c.run().any()
    c.scale[0] = 0.0
    c.scale[1] = 1.0
    c.check(c.run())           # all scores equal


def test_attention_far_offsets(kv):
    # a cache of over 2^32 bytes a side, its last pages used
    hk, dim = 8, 128
    pages = 70000
    small = AttnCase(kv, [(4, 700)], 16, hk, dim, 12, extra_pages=0)
    n = small.codes.shape[1]
    cache = kv.KvCache(torch.zeros(pages, hk, dim // 16, PAGE, 16, dtype=torch.float8_e4m3fn, device="cuda"),
                       torch.zeros(pages, hk, dim, PAGE, dtype=torch.float8_e4m3fn, device="cuda"),
                       torch.ones(pages, hk, device="cuda"), torch.ones(pages, hk, device="cuda"))
    part = small.device()
    for a, b in ((cache.k, part.k), (cache.v, part.v)):
        a.view(torch.uint8)[pages - n:] = b.view(torch.uint8)
    cache.k_scale[pages - n:] = part.k_scale
    cache.v_scale[pages - n:] = part.v_scale
    clean = small.run()
    small.table = np.where(small.table >= 0, small.table + pages - n, small.table)
    assert np.array_equal(small.run(cache), clean)
    # and an append to the last page
    q = dev(small.q.reshape(4, -1))
    x = torch.cat([q, torch.ones(4, 2 * hk * dim, dtype=torch.float16, device="cuda")], 1)
    kv.rope_append(cache, x, 16, i32([0] * 4), i32([pages * PAGE - 4 + i for i in range(4)]), None)
    torch.cuda.synchronize()
    tail = kv_ref.unpack_v(bytes_of(cache.v[pages - 1:]))
    assert np.array_equal(kv_ref.VALUES[tail[0, :, 60:]] * host(cache.v_scale[-1])[:, None, None], np.ones((hk, 4, dim)))


def test_attention_strides_scratch_streams(kv):
    c = AttnCase(kv, [(8, 3000), (1, 200)], 10, 2, 128, 13)
    ref = c.run()
    c.check(ref)
    cache, n = c.device(), 9
    row_start, seq, table = i32(c.row_start), i32(c.seq), i32(c.table)
    wide = torch.zeros(n, 10 * 128 + 40, dtype=torch.float16, device="cuda")
    q = wide[:, 16:16 + 1280]
    q[:] = dev(c.q.reshape(n, -1))
    out = torch.zeros(n, 1280 + 12, dtype=torch.float16, device="cuda")[:, 4:1284]
    tw = torch.full((2, c.width + 5), -1, dtype=torch.int32, device="cuda")
    tw[:, :c.width] = table
    kv.attention(cache, q, row_start, seq, tw[:, :c.width], 8, out=out)
    assert np.array_equal(host(out).reshape(ref.shape), ref)
    # any hint of the rows, any scratch: the same to rounding
    need = kv.attention_scratch_bytes(2, 8, 10, 2, 128, c.width)
    for most in (0, 1, 3, 100):
        for size in (0, kv.SCRATCH_ZEROED, kv.SCRATCH_ZEROED + 30000, need // 2, need):
            s = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
            s[kv.SCRATCH_ZEROED:] = 255
            y = kv.attention(cache, q, row_start, seq, table, most, scratch_=s[:size] if size else s[:0])
            c.check(host(y).reshape(ref.shape).astype(np.float64))
            assert int(s[:kv.SCRATCH_ZEROED].count_nonzero()) == 0
    # another stream, several in a row; bit for bit
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        y = kv.attention(cache, q, row_start, seq, table, 8, stream=side)
        side.synchronize()
        assert np.array_equal(host(y).reshape(ref.shape), ref)


# ---------------------------------------------------------------- verify_sampled

def verify_case(kv, counts, n, seed, sampled, temperature=0.8, edit=None, stride=0, stream=None):
    rng = np.random.default_rng(seed)
    rows = max(1, sum(counts))
    start = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    logits = (2.5 * rng.standard_normal((rows, n))).astype(np.float16)
    near = (logits + 0.7 * rng.standard_normal((rows, n))).astype(np.float16)
    draft = near if sampled else None
    noise = temperature * rng.gumbel(size=(rows, n)) if sampled else 0.0
    picked = (near + noise).argmax(1)
    tokens = np.concatenate([[0], picked[:-1]])
    u, su = rng.random(rows).astype(np.float32), rng.random(len(counts)).astype(np.float32)
    if edit:
        edit(logits, draft, tokens, u, su)

    def wide(x):
        if x is None:
            return None
        t = torch.full((rows, n + stride), 9.0, dtype=torch.float16, device="cuda")
        t[:, :n] = dev(x)
        return t[:, :n]
    args = (wide(logits), i32(tokens), i32(start), dev(u), dev(su), wide(draft), temperature)
    log(f"verify {counts[:8]} of {n} sampled {sampled} seed {seed}")
    torch.cuda.synchronize()
    got = kv.verify_sampled(*args, stream=stream)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore", divide="ignore"):
        ref = kv_ref.verify(logits, draft, tokens, start, 1.0 / temperature, u, su)
    return [host(g) for g in got], ref, args


def check_verify(got, ref):
    assert got[0].tolist() == list(ref[0]) and got[1].tolist() == list(ref[1])
    assert (np.abs(got[2] - ref[2]) <= 2.0 ** -23 * ref[2] + 1e-10).all()


@pytest.mark.parametrize("counts", [[1], [8], [2], [3, 0, 1, 8, 5], [1] * 40, [17, 2]])
@pytest.mark.parametrize("n", [1, 2, 7, 1000, 4089, 4096, 5001, 151936])
@pytest.mark.parametrize("sampled", [False, True])
def test_verify(kv, counts, n, sampled):
    if n == 151936 and len(counts) > 5:
        counts = counts[:3]
    got, ref, _ = verify_case(kv, counts, n, n + len(counts), sampled)
    check_verify(got, ref)


@pytest.mark.parametrize("temperature", [0.05, 0.3, 1.7, 30.0])
def test_verify_temperatures(kv, temperature):
    for seed in range(4):
        got, ref, _ = verify_case(kv, [8, 4], 3001, seed, seed % 2 == 0, temperature)
        check_verify(got, ref)


def test_verify_every_accept_length(kv):
    for n_ok in range(8):
        def edit(logits, draft, tokens, u, su):
            u[:] = 0.0
            if n_ok < 7:
                u[n_ok] = 1.0            # never below p / q of a draft the target likes less
                logits[n_ok, tokens[n_ok + 1]] = -20
        got, ref, _ = verify_case(kv, [8], 2000, n_ok, False, edit=edit)
        check_verify(got, ref)
        assert got[0].tolist() == [n_ok]


def test_verify_odd_rows_and_strides(kv):
    # rows that begin anywhere in a 16-byte granule
    for stride in (0, 1, 3, 8):
        for n in (4095, 333):
            got, ref, _ = verify_case(kv, [5, 3], n, stride, True, stride=stride)
            check_verify(got, ref)


def test_verify_masked_logits(kv):
    # -inf and the type's lowest value as masks: no weight there, in either distribution
    def edit(logits, draft, tokens, u, su):
        allowed = np.zeros(logits.shape[1], bool)
        allowed[100:140] = True
        logits[:, ~allowed] = -np.inf
        logits[1, ~allowed] = np.finfo(np.float16).min
        draft[:, ~allowed] = -np.inf
        tokens[1:] = 100 + tokens[1:] % 40
    for seed in range(6):
        got, ref, _ = verify_case(kv, [4, 4], 9000, seed, True, edit=edit)
        check_verify(got, ref)
        assert ((got[1] >= 100) & (got[1] < 140)).all()


def test_verify_random_numbers_at_their_ends(kv):
    for value in (0.0, float(np.nextafter(np.float32(1), np.float32(0)))):
        def edit(logits, draft, tokens, u, su):
            su[:] = value
        for sampled in (False, True):
            got, ref, _ = verify_case(kv, [3, 1], 5000, 3, sampled, edit=edit)
            check_verify(got, ref)


def test_verify_same_distributions_accept_all(kv):
    def edit(logits, draft, tokens, u, su):
        draft[:] = logits
        u[:] = np.nextafter(np.float32(1), np.float32(0))
    got, _, _ = verify_case(kv, [8], 5000, 4, True, edit=edit)
    assert got[0].tolist() == [7] and (got[2][:7] == 1.0).all()


def test_verify_bad_rows_and_tokens(kv):
    n = 5000

    def bad_draft(logits, draft, tokens, u, su):
        tokens[2] = n
        tokens[6] = -1
    for sampled in (False, True):
        got, ref, _ = verify_case(kv, [4, 4], n, 5, sampled, edit=bad_draft)
        check_verify(got, ref)
        assert got[2][1] == 0.0 and got[2][5] == 0.0
    for value in (np.nan, np.inf):
        def bad_logit(logits, draft, tokens, u, su):
            logits[0, 4321] = value
            u[4:] = 0
            logits[7, 17] = value
        got, _, _ = verify_case(kv, [4, 4], n, 6, False, edit=bad_logit)
        assert got[0].tolist()[0] == 0 and got[1].tolist()[0] == -1 and np.isnan(got[2][0])
        assert got[0].tolist()[1] < 3 or got[1].tolist()[1] == -1

    def nothing(logits, draft, tokens, u, su):
        logits[0, :] = -np.inf
    got, _, _ = verify_case(kv, [2], n, 7, False, edit=nothing)
    assert got[0].tolist() == [0] and got[1].tolist() == [-1] and np.isnan(got[2][0])

    def bad_draft_row(logits, draft, tokens, u, su):
        draft[0, 99] = np.nan
    got, _, args = verify_case(kv, [2], n, 8, True, edit=bad_draft_row)
    p = kv_ref.softmax(host(args[0])[0].astype(np.float64) / 0.8)   # drawn from the target alone
    want = int((np.cumsum(p) <= float(host(args[4])[0])).sum())
    assert got[0].tolist() == [0] and got[1].tolist() == [want] and np.isnan(got[2][0])
    # row_start out of order, or past the rows
    a = list(args)
    a[2] = i32([5, 1])
    got = kv.verify_sampled(*a)
    assert host(got[0]).tolist() == [0] and host(got[1]).tolist() == [-1]
    a[2] = i32([0, 900])
    got = kv.verify_sampled(*a)
    assert host(got[0]).tolist() == [0] and host(got[1]).tolist() == [-1]


def test_verify_repeats_and_streams(kv):
    got, ref, args = verify_case(kv, [8] * 6, 20000, 9, True)
    check_verify(got, ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side, None):
        again = kv.verify_sampled(*args, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(again, got):
            assert np.array_equal(host(a), b)
    for s in kv._scratches.values():
        assert int(s[:kv.SCRATCH_ZEROED].count_nonzero()) == 0


# ---------------------------------------------------------------- together

def test_round_in_a_graph(kv):
    # plan, append, attention and verification captured once and replayed with eager work between:
    # every replay gives the eager round's bits
    rng = np.random.default_rng(20)
    lens, hq, hk, dim, n = [(8, 700), (3, 100)], 10, 2, 128, 6000
    c = AttnCase(kv, [(0, t - r) for r, t in lens], hq, hk, dim, 21, extra_pages=6)
    rows = sum(r for r, _ in lens)
    before, add = i32([t - r for r, t in lens]), i32([r for r, _ in lens])
    held = i32([-(-(t - r) // PAGE) for r, t in lens])
    width = c.width + 2
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    table[:, :c.width] = i32(np.clip(c.table, 0, None))
    used = set(int(x) for r in range(2) for x in c.table[r, :-(-(lens[r][1] - lens[r][0]) // PAGE)])
    free = i32([p for p in range(c.codes.shape[1]) if p not in used])
    count = i32([len(free)])
    qkv = dev((rng.standard_normal((rows, (hq + 2 * hk) * dim))).astype(np.float16))
    w = dev((1 + 0.1 * rng.standard_normal(dim)).astype(np.float16))
    f = dev((1e4 ** (-np.arange(64) / 64)).astype(np.float32))
    logits = dev((2 * rng.standard_normal((rows, n))).astype(np.float16))
    tokens, u, su = i32(rng.integers(0, n, rows)), dev(rng.random(rows).astype(np.float32)), dev(rng.random(2).astype(np.float32))

    def step(cache, out):
        r = kv.plan_round(before, add, held, table, free, count, out=out[0])
        q = kv.rope_append(cache, qkv, hq, r.positions, r.slots, f, w, w, out=out[1])
        y = kv.attention(cache, q, r.row_start, r.seq_lens, table, 8, out=out[2])
        v = kv.verify_sampled(logits, tokens, r.row_start, u, su, out=out[3])
        return [r.slots, r.seq_lens, q, y, *v, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale]

    def outs():
        z = lambda *s, t=torch.float16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        return (kv.Round.empty(2, rows), z(rows, hq * dim), z(rows, hq * dim),
                (z(2, t=torch.int32), z(2, t=torch.int32), z(rows, t=torch.float32)))
    log("round in a graph")
    want = [host(t) for t in step(c.device(), outs())]
    cache, out = c.device(), outs()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(c.device(), outs())        # this stream's scratch exists before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(cache, out)
    fresh = c.device()
    for _ in range(4):
        for a, b in zip((cache.k, cache.v), (fresh.k, fresh.v)):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        cache.k_scale.copy_(fresh.k_scale)
        cache.v_scale.copy_(fresh.v_scale)
        for t in got[:-3]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, e in zip(got, want):
            assert np.array_equal(host(g), e, equal_nan=g.is_floating_point())
        step(c.device(), outs())
        torch.cuda.synchronize()
