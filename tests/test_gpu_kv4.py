"""GPU parity of the 4-bit KV cache's operators against plain FP64 references (kv4_ref.py).

Tolerances, derived before the first run:
  queries of rope_append   as over the 8-bit cache (test_gpu_kv.py);
  codes and scales         the values they stand for equal (keys are computed in 64 bits; seeds are fixed);
  read                     code * scale exact, times the unit in FP32 (2^-24), rounded to FP16: 2^-11 + 2^-23 of the
                           value, or 2^-25 among FP16's subnormal numbers; units that are powers of two: equal;
  attention                2^-11 |y| (output) + 2^-11 a (each weight rounded to FP16) +
                           2^-24 (dim s + tokens) a (FP32 scores up to s = 40 and sums), a = sum w |v| / sum w,
                           + tokens 2^-25 max |v| (weights below FP16's normal range, the largest being
                           at least 1) + 2^-25.
"""
import threading

import numpy as np
import pytest
import torch

import kv4_ref
import kv_ref
from gpu_util import dev, host, log, need_gpu
from test_gpu_kv import RAGGED, AttnCase, i32, run_slots

pytestmark = pytest.mark.gpu
PAGE = kv4_ref.PAGE


@pytest.fixture(scope="module")
def kv():
    need_gpu()
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def device_cache(kv, codes, scales, units):
    """A KvCache4 of codes [2, pages, heads, 64, dim], scale codes and units [2, heads]."""
    _, pages, heads, _, dim = codes.shape
    (k, ks), (v, vs) = (kv4_ref.pack(codes[i], scales[i], kind) for i, kind in enumerate("kv"))
    shape = (pages, heads, dim // 32, PAGE, 16)
    return kv.KvCache4(dev(k.reshape(shape)), dev(v.reshape(shape)),
                       dev(ks.reshape(pages, heads, PAGE, dim // 16)).view(torch.float8_e4m3fn),
                       dev(vs.reshape(pages, heads, dim // 64, 16, 16)).view(torch.float8_e4m3fn),
                       dev(np.asarray(units[0], np.float32)), dev(np.asarray(units[1], np.float32)))


def host_cache(cache):
    u8 = lambda t: host(t.view(torch.uint8))  # noqa: E731
    k, ks = kv4_ref.unpack(host(cache.k), u8(cache.k_scale), cache.dim, "k")
    v, vs = kv4_ref.unpack(host(cache.v), u8(cache.v_scale), cache.dim, "v")
    return np.stack([k, v]), np.stack([ks, vs])


def random_cache(rng, pages, heads, dim):
    return (rng.integers(0, 16, (2, pages, heads, PAGE, dim)).astype(np.uint8),
            rng.integers(0x20, 0x48, (2, pages, heads, PAGE, dim // 16)).astype(np.uint8))


# ---------------------------------------------------------------- rope_append

def append_case(kv, dim, hq, hk, slots, positions, pages, seed, rot=None, interleaved=False, norm=True, x=None,
                stride=0, inplace=False, units=None, stream=None):
    rng = np.random.default_rng(seed)
    rows, rot = len(slots), dim if rot is None else rot
    if x is None:
        x = (rng.standard_normal((rows, (hq + 2 * hk) * dim)) * 10.0 ** rng.uniform(-1, 1, (rows, 1))).astype(np.float16)
    qw, kw = ((1 + 0.3 * rng.standard_normal((2, dim))).astype(np.float16) if norm else (None, None))
    f = (1e6 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    codes, scales = random_cache(rng, pages, hk, dim)
    units = np.full((2, hk), 0.125, np.float32) if units is None else np.asarray(units, np.float32)
    cache = device_cache(kv, codes, scales, units)
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
    want, ws = codes.copy(), scales.copy()
    for i, new in enumerate((k_ref, xs[:, hq + hk:])):
        kv4_ref.append(want[i], ws[i], new, units[i], slots)
    got = host(q).astype(np.float64)
    length = np.abs(q_ref).reshape(rows, hq, dim).max(-1).repeat(dim, 1).reshape(rows, -1)
    ok = np.isfinite(q_ref)
    assert np.array_equal(np.isnan(got), np.isnan(q_ref))
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - q_ref) <= 2.0 ** -11 * np.abs(q_ref) + 2.0 ** -17 * length + 2.0 ** -25)[ok].all()
    gc, gs = host_cache(cache)
    for i, kind in enumerate("kv"):
        assert np.array_equal(gs[i], ws[i]), f"{(gs[i] != ws[i]).sum()} scales of {kind} differ"
        same = kv4_ref.E2M1[gc[i]] == kv4_ref.E2M1[want[i]]       # (a zero has two codes)
        assert same.all(), f"{(~same).sum()} codes of {kind} differ"
    return cache, want, ws


@pytest.mark.parametrize("dim,hq,hk", [(128, 40, 8), (64, 4, 4), (256, 8, 1), (128, 10, 2), (64, 64, 1), (256, 6, 3),
                                       (64, 18, 9)])
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
    slots, pos = run_slots([(37 * i % 500, 1 + i % 4) for i in range(200)], 420, 2)
    append_case(kv, 128, 40, 8, slots, pos, 420, 3)


def test_append_slots_in_any_order(kv):
    # rows of one page scattered over the call, one slot several times (far apart too), padding, slots out of range
    rng = np.random.default_rng(5)
    slots = [7] + list(rng.permutation(3 * PAGE)[:70]) + [-1, 7, 7, -5, 4 * PAGE, 2 ** 31 - 1, -2 ** 31, 7]
    append_case(kv, 64, 4, 2, slots, rng.integers(0, 900, len(slots)), 4, 6)
    slots = list(range(300)) + [5] * 200 + [299, 0]
    append_case(kv, 128, 2, 1, slots, np.arange(502), 5, 7)


@pytest.mark.parametrize("rows", [2, 63, 1025, 2300])
def test_append_a_slot_taken_again(kv, rows):
    rng = np.random.default_rng(rows)
    slots = rng.permutation(40 * PAGE)[:rows].astype(np.int32)
    first = rng.permutation(rows - 1)[:rows // 3 + 1]
    for i in first:                                  # at any distance, also more than once
        slots[rng.integers(i + 1, rows)] = slots[i]
    slots[-1] = slots[0]
    append_case(kv, 64, 2, 1, slots, rng.integers(0, 5000, rows), 40, rows)


@pytest.mark.parametrize("unit", [2.0 ** -30, 2.0 ** -6, 0.7, 3.0e-3, 1000.0, 1e30])
def test_append_units(kv, unit):
    # values far above what the unit holds (they saturate), of its size, far below (coarse scales, zeros), no power of two
    slots, pos = run_slots([(60, 3), (33, 1), (50, 30)], 6, 3)
    append_case(kv, 128, 4, 2, slots, pos, 6, 8, units=[[unit, unit * 1.37], [unit, 0.125]])


@pytest.mark.parametrize("unit", [0.0, -1.0, np.inf, -np.inf, np.nan])
def test_append_units_that_are_none(kv, unit):
    # such a head's groups read as NaN; the other head's are as ever
    slots, pos = run_slots([(60, 6)], 3, 3)
    append_case(kv, 64, 4, 2, slots, pos, 3, 9, units=[[unit, 0.25], [0.25, unit]])


@pytest.mark.parametrize("unit", [0.125, 0.0859375, 0.77, 1.0 / 3])
def test_append_ties(kv, unit):
    # values halfway between two codes, and largest ones halfway between two scales, exactly in 64 bits
    # where the unit allows it, a step of FP16 to either side elsewhere
    u = float(np.float32(unit))
    rng = np.random.default_rng(12)
    rows, hq, hk, dim = 40, 2, 1, 128
    x = np.zeros((rows, (hq + 2 * hk) * dim))
    v = x[:, (hq + hk) * dim:].reshape(rows, dim // 16, 16)
    mids = (kv_ref.VALUES[1:127] + kv_ref.VALUES[:126]) / 2
    for r in range(rows):
        for g in range(dim // 16):
            scale = kv_ref.VALUES[rng.integers(1, 0x50)]
            v[r, g, 0] = rng.choice(mids[:0x50]) * 6 * u if r % 2 else scale * 6 * u
            v[r, g, 1:8] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]) * scale * u
            v[r, g, 8:15] = -v[r, g, 1:8] * (1 + rng.choice([0, 2.0 ** -10, -2.0 ** -10], 7))
    x[:, hq * dim:(hq + hk) * dim] = x[:, (hq + hk) * dim:]
    append_case(kv, dim, hq, hk, list(range(rows)), [0] * rows, 1, 13, rot=0, norm=False, x=x.astype(np.float16),
                units=[[u], [u]])


def test_append_special_values(kv):
    rows, hq, hk, dim = 6, 4, 2, 64
    x = np.random.default_rng(9).standard_normal((rows, (hq + 2 * hk) * dim)).astype(np.float16)
    x[1, :] = 0.0                          # a row of zeros
    x[2, (hq + hk) * dim + 3] = np.inf     # an infinite value makes its group NaN
    x[3, (hq + hk) * dim + 20] = np.nan    # and so does NaN
    x[4, hq * dim + 5] = np.nan            # a NaN key makes its whole head NaN when normed, its group and its partner's else
    x[5, :] = 6e-8                         # FP16 subnormals
    append_case(kv, dim, hq, hk, [0, 1, 2, 3, 4, 5], [9, 8, 7, 6, 5, 4], 2, 10, x=x)
    append_case(kv, dim, hq, hk, [70, 71, 72, 73, 74, 75], [9, 8, 7, 6, 5, 4], 2, 10, x=x, norm=False)
    append_case(kv, dim, hq, hk, [0] + [-1] * 5, [0] * 6, 1, 11, x=np.zeros_like(x))


def test_append_strides_in_place_and_streams(kv):
    slots, pos = run_slots([(4090, 8)], 4, 4)
    append_case(kv, 128, 10, 2, slots, pos, 4, 12, stride=24)
    append_case(kv, 128, 10, 2, slots, pos, 4, 13, inplace=True)
    append_case(kv, 128, 10, 2, slots, pos, 4, 14, stream=torch.cuda.Stream())


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 5), (128, 8), (128, 3), (256, 2)])
@pytest.mark.parametrize("unit", [0.125, 0.3, 40.0])
def test_read(kv, dim, heads, unit):
    rng = np.random.default_rng(dim + heads)
    codes, scales = random_cache(rng, 5, heads, dim)
    scales[:, 1] = rng.integers(0, 0x7F, scales[:, 1].shape)       # the whole range, and beyond FP16's with unit 40
    scales[:, 2, :, 7] = 0x7F
    units = unit * np.array([1.0, 2.0])[:, None] * np.ones(heads)
    cache = device_cache(kv, codes, scales, units)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale.view(torch.uint8), cache.v_scale.view(torch.uint8))]
    want = [kv4_ref.values(codes[i], scales[i], np.float32(units[i])) for i in range(2)]
    for slots in ([0], [63], [64 * 5 - 1], list(rng.permutation(5 * PAGE)), [7] * 20 + [-1, 64 * 5, 3, -2 ** 31, 2 ** 31 - 1],
                  list(range(130, 205))):
        log(f"read dim {dim} heads {heads} rows {len(slots)}")
        got = kv.read(cache, i32(slots))
        for g, w in zip(got, want):
            ref = np.zeros((len(slots), heads, dim))
            for t, s in enumerate(slots):
                if 0 <= s < 5 * PAGE:
                    ref[t] = w[s // PAGE, :, s % PAGE]
            y = host(g).astype(np.float64).reshape(ref.shape)
            assert np.array_equal(np.isnan(y), np.isnan(ref))
            if unit == 0.125:
                with np.errstate(over="ignore"):
                    assert np.array_equal(y, ref.astype(np.float16).astype(np.float64), equal_nan=True)
            else:
                big = np.abs(ref) > 65519
                assert np.isinf(y[big]).all()
                ok = ~big & ~np.isnan(ref)
                assert (np.abs(y - ref)[ok] <= np.maximum((2.0 ** -11 + 2.0 ** -23) * np.abs(ref), 2.0 ** -25)[ok]).all()
    for a, b in zip(before, (cache.k, cache.v, cache.k_scale.view(torch.uint8), cache.v_scale.view(torch.uint8))):
        assert torch.equal(a, b)


def test_read_strides_streams_and_units(kv):
    rng = np.random.default_rng(3)
    codes, scales = random_cache(rng, 3, 2, 128)
    cache = device_cache(kv, codes, scales, [[0.125, np.nan], [-1.0, 0.5]])
    slots = i32(list(range(100)) + [-1])
    wide = torch.full((2, 101, 256 + 24), 9.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    out = kv.read(cache, slots, out=(wide[0, :, 8:264], wide[1, :, 16:272]), stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    k, v = (host(t).astype(np.float64) for t in out)
    assert np.isnan(k[:100, 128:]).all() and np.isnan(v[:100, :128]).all() and not k[100].any() and not v[100].any()
    assert np.array_equal(k[:100, :128], kv4_ref.values(codes[0], scales[0], [0.125, 1])[:, 0].reshape(-1, 128)[:100])
    assert (wide[0, :, :8] == 9).all() and (wide[0, :, 264:] == 9).all() and (wide[1, :, :16] == 9).all()


# ---------------------------------------------------------------- attention

class AttnCase4(AttnCase):
    def __init__(self, kv, lens, hq, hk, dim, seed, extra_pages=2, size=2.0):
        super().__init__(kv, lens, hq, hk, dim, seed, extra_pages, size)
        rng = np.random.default_rng(seed + 1000)
        self.codes, self.scale = random_cache(rng, self.codes.shape[1], hk, dim)    # scales 2^-3 .. 2^1.9
        self.units = np.float32(2.0) ** rng.integers(-3, 1, (2, hk)) * np.float32(1.1)

    def values(self):
        return tuple(kv4_ref.values(self.codes[i], self.scale[i], self.units[i]) for i in range(2))

    def device(self):
        return device_cache(self.kv, self.codes, self.scale, self.units)


@pytest.mark.parametrize("dim,hq,hk", [(128, 40, 8), (128, 5, 1), (64, 8, 8), (64, 16, 1), (256, 8, 2), (128, 6, 2), (256, 2, 2)])
@pytest.mark.parametrize("rows,tokens", [(1, 1), (1, 63), (1, 64), (1, 65), (8, 8), (8, 200), (3, 1000), (8, 4099), (1, 3001)])
def test_attention(kv, dim, hq, hk, rows, tokens):
    c = AttnCase4(kv, [(rows, tokens)], hq, hk, dim, dim + tokens)
    c.check(c.run())


@pytest.mark.parametrize("dim,hq,hk,rows,tokens", [(128, 40, 8, 256, 700), (64, 4, 1, 100, 1000), (256, 4, 2, 70, 300),
                                                   (128, 16, 2, 33, 64), (128, 8, 8, 64, 2048), (64, 2, 2, 300, 5000)])
def test_attention_prompt_blocks(kv, dim, hq, hk, rows, tokens):
    c = AttnCase4(kv, [(rows, max(rows, tokens))], hq, hk, dim, rows)
    c.check(c.run())


@pytest.mark.parametrize("dim,hq,hk", [(128, 10, 2), (64, 4, 4), (256, 16, 1)])
@pytest.mark.parametrize("window", [0, 1, 64, 100, 5000])
def test_attention_ragged_and_windows(kv, dim, hq, hk, window):
    c = AttnCase4(kv, RAGGED, hq, hk, dim, 5)
    c.check(c.run(window=window), window)


# so many requests that the row tiles of a KV head stay together: two and three tiles, some pieces cut
MANY = [(1 + (i * 5) % 8, 8 + (i * 397) % 1500) for i in range(19)] + [(8, 2600)]


@pytest.mark.parametrize("dim,hq,hk", [(128, 15, 3), (64, 12, 3), (128, 16, 4), (64, 30, 6)])
@pytest.mark.parametrize("window", [0, 1, 70, 1000])
def test_attention_tiles_together(kv, dim, hq, hk, window):
    c = AttnCase4(kv, MANY, hq, hk, dim, 16)
    clean = c.run(window=window)
    c.check(clean, window)
    # NaN in the unseen, and a value group that only later rows of the last request see
    used = np.zeros(c.codes.shape[1:4], bool)
    for r, (n, t) in enumerate(c.lens):
        for j in range(max(0, t - n + 1 - window) if window else 0, t):
            used[c.table[r, j // PAGE], :, j % PAGE] = True
    c.scale[:, ~used] = 0x7F
    assert np.array_equal(c.run(window=window), clean)
    c.scale[1, c.table[-1, 2595 // PAGE], 1, 2595 % PAGE, 2] = 0x7F
    y = c.run(window=window)
    group, hit = hq // hk, np.zeros(y.shape, bool)
    hit[-5:, group:2 * group, 32:48] = True
    if window == 1:
        hit[-4:] = False
    assert np.array_equal(np.isnan(y), hit) and np.array_equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("window", [0, 77])
def test_attention_ragged_many_rows(kv, window):
    c = AttnCase4(kv, [(70, 300), (1, 1), (0, 40), (200, 210), (33, 64), (100, 1300)], 6, 2, 128, 15)
    c.check(c.run(window=window), window)


def test_attention_many_requests(kv):
    lens = [(1 + i % 3, 3 + (i * 97) % 700) for i in range(300)]
    c = AttnCase4(kv, lens, 4, 2, 64, 6)
    c.check(c.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [6, 70])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_unseen_tokens_never_matter(kv, dim, rows, window):
    # NaN scales, the largest and negative ones, and any codes in everything that no row may see; NaN scales of
    # tokens that only later rows see reach those rows alone, and of values only their group
    c = AttnCase4(kv, [(rows, 150), (2, 64), (4, 321)], 4, 2, dim, 7)
    clean = c.run(window=window)
    c.check(clean, window)
    used = np.zeros(c.codes.shape[1:4], bool)
    for r, (n, t) in enumerate(c.lens):
        for j in range(max(0, t - n + 1 - window) if window else 0, t):
            used[c.table[r, j // PAGE], :, j % PAGE] = True
    for junk in (0x7F, 0xFF, 0x7E, 0xFE):
        keep = c.codes.copy(), c.scale.copy()
        c.scale[:, ~used] = junk
        c.codes[:, ~used] = junk & 15
        assert np.array_equal(c.run(window=window), clean), hex(junk)
        c.codes, c.scale = keep
    # request 0, KV head 1: the value of a row's own token, a group in the middle
    i, group = rows - 3, dim // 16 - 2
    p = 150 - rows + i
    c.scale[1, c.table[0, p // PAGE], 1, p % PAGE, group] = 0x7F
    y = c.run(window=window)
    hit = np.zeros(y.shape, bool)
    hit[i:rows, 2:4, 16 * group:16 * group + 16] = True
    assert np.array_equal(np.isnan(y), hit)
    assert np.array_equal(y[~hit], clean[~hit])
    # and a NaN key group makes the whole of those rows NaN
    c.scale[0, c.table[0, p // PAGE], 1, p % PAGE, 1] = 0xFF
    y = c.run(window=window)
    hit[i:rows, 2:4, :] = True
    assert np.array_equal(np.isnan(y), hit)
    assert np.array_equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,tokens", [(5, 700), (80, 700)])
def test_attention_nan_groups_that_all_rows_see(kv, dim, rows, tokens):
    c = AttnCase4(kv, [(rows, tokens)], 4, 2, dim, 17)
    clean = c.run()
    c.scale[1, c.table[0, 2], 0, 11, 1] = 0x7F      # page 2 of 11: in the middle of some piece
    y = c.run()
    hit = np.zeros(y.shape, bool)
    hit[:, :2, 16:32] = True
    assert np.array_equal(np.isnan(y), hit) and np.array_equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("rows", [5, 80])
def test_attention_units_that_are_none(kv, rows):
    c = AttnCase4(kv, [(rows, 300), (2, 0)], 6, 3, 64, 18)
    clean = c.run()
    for unit in (0.0, -1.0, np.inf, np.nan):
        for side in (0, 1):
            keep = c.units.copy()
            c.units[side, 1] = unit
            y = c.run()
            c.units = keep
            assert np.isnan(y[:rows, 2:4]).all() and not y[rows:].any()      # (what sees nothing is zeros)
            assert np.array_equal(y[:, [0, 1, 4, 5]], clean[:, [0, 1, 4, 5]])


def test_attention_rows_that_see_nothing(kv):
    # fewer tokens than rows: the first rows stand before the first token
    for lens in ([(5, 3), (4, 0), (2, 100), (3, 1)], [(70, 3), (60, 0), (50, 100), (90, 70)], [(300, 200)]):
        c = AttnCase4(kv, lens, 8, 2, 64, 8)
        y = c.run()
        c.check(y)
        for w in (2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30):
            assert np.array_equal(c.run(window=w), y)
        at = 0
        for n, t in lens:
            assert not y[at:at + max(n - t, 0)].any()
            at += n
    c = AttnCase4(kv, [(5, 3), (4, 0), (2, 100), (3, 1)], 8, 2, 64, 8)
    c.seq = [-4, -2 ** 31, 100, 1]
    y = c.run()
    assert not y[:9].any() and y[9:11].any()


def test_attention_bad_pages_and_lengths(kv):
    c = AttnCase4(kv, [(2, 200), (3, 200), (2, 90)], 8, 2, 64, 9)
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


@pytest.mark.parametrize("rows,page", [(100, 0), (100, 1), (200, 2)])
def test_attention_bad_pages_many_rows(kv, rows, page):
    # a page that only the later rows see
    tokens = 64 * 3
    c = AttnCase4(kv, [(rows, tokens)], 4, 2, 128, 19)
    clean = c.run()
    c.table[0, page] = -1
    y = c.run()
    first = max(0, 64 * page - (tokens - rows))
    assert np.isnan(y[first:]).all() and np.array_equal(y[:first], clean[:first])


@pytest.mark.parametrize("rows", [3, 90])
def test_attention_long_tables_in_one_piece(kv, rows):
    # page numbers are loaded 64 at a time: bad ones around the ends of those, with segments whole (no scratch)
    tokens = 64 * 133 + 5
    c = AttnCase4(kv, [(rows, tokens)], 4, 1, 64, 23)
    c.check(c.run())
    cache, none = c.device(), torch.zeros(0, dtype=torch.uint8, device="cuda")
    args = dev(c.q.reshape(rows, -1)), i32(c.row_start), i32(c.seq)
    y = host(kv.attention(cache, *args, i32(c.table), rows, scratch_=none)).reshape(c.q.shape)
    c.check(y.astype(np.float64))
    for page in (0, 1, 62, 63, 64, 65, 127, 128, 132):
        bad = c.table.copy()
        bad[0, page] = -1
        got = host(kv.attention(cache, *args, i32(bad), rows, scratch_=none))
        sees = np.arange(tokens - rows, tokens) >= 64 * page     # (the last page is behind the first rows)
        assert np.isnan(got[sees]).all() and np.isfinite(got[~sees]).all(), page
        # in a window: NaN in the rows for which the page's last token is not behind it, and the others as if
        # the page were there
        window = 64 * (132 - page)
        if window > 0:
            good, got = (host(kv.attention(cache, *args, i32(t), rows, window=window, scratch_=none))
                         for t in (c.table, bad))
            sees = np.arange(tokens - rows, tokens) - window < 64 * page + 63
            assert np.isnan(got[sees]).all() and np.array_equal(got[~sees], good[~sees]), page


@pytest.mark.parametrize("dim,hq,hk", [(64, 4, 2), (128, 2, 2), (256, 8, 1)])
@pytest.mark.parametrize("rows,tokens", [(8, 6), (100, 90), (200, 256), (200, 300)])
def test_attention_more_rows_than_the_table_has_places(kv, dim, hq, hk, rows, tokens):
    width = -(-tokens // PAGE) - 1                 # 0 pages for 6 tokens, 1 for 90, 3 and 4
    c = AttnCase4(kv, [(2, PAGE * max(width, 1)), (rows, tokens), (1, 5)], hq, hk, dim, 50)
    c.table = c.table[:, :width]
    if width == 0:
        c.seq = [0, tokens, -3]
    y = c.run()
    assert np.isnan(y[2:2 + rows]).all()
    if width == 0:
        assert not y[:2].any() and not y[2 + rows:].any()
    else:
        assert np.isfinite(y[:2]).all() and np.isfinite(y[2 + rows:]).all()


def test_attention_infinite_queries(kv):
    for rows in (3, 70):
        c = AttnCase4(kv, [(rows, 100)], 4, 1, 64, 10)
        clean = c.run()
        c.q[1, 2, 5] = np.inf
        c.q[2, 0, 0] = np.nan
        y = c.run()
        hit = np.zeros(y.shape, bool)
        hit[1, 2] = hit[2, 0] = True
        assert np.isnan(y[hit]).all() or not np.isfinite(y[1, 2]).all()
        assert np.array_equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("rows", [8, 90])
def test_attention_peaked_scores_and_scales(kv, rows):
    # scores up to +-40 (one token takes all, wherever it lies); value scales over their whole range; zeros
    c = AttnCase4(kv, [(rows, 1500)], 10, 2, 128, 11, size=2.0)
    k = c.values()[0][c.table[0, :24]].transpose(1, 0, 2, 3).reshape(2, -1, 128)[:, :1500 - rows]
    s = max(np.abs(k[h // 5] @ c.q[:, h].T.astype(np.float64)).max() for h in range(10)) * 128 ** -0.5
    c.q = (c.q.astype(np.float64) * 39 / s).astype(np.float16)
    c.check(c.run())
    c.scale[1] = np.random.default_rng(0).integers(0, 0x7F, c.scale[1].shape)
    c.check(c.run())
    c.scale[1] = 0
    assert not c.run().any()
    c.scale[0] = 0
    c.scale[1] = 0x38
    c.check(c.run())           # all scores equal


def test_attention_far_offsets(kv):
    # codes of over 2^32 bytes a side, the last pages used by every operator
    hk, dim = 8, 256
    pages = 70000
    small = AttnCase4(kv, [(4, 700)], 16, hk, dim, 12, extra_pages=0)
    n = small.codes.shape[1]
    cache = kv.KvCache4.empty(pages, hk, dim)
    part = small.device()
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(cache, name).view(torch.uint8)[pages - n:] = getattr(part, name).view(torch.uint8)
    cache.k_unit, cache.v_unit = part.k_unit, part.v_unit
    clean = small.run()
    small.table = np.where(small.table >= 0, small.table + pages - n, small.table)
    assert np.array_equal(small.run(cache), clean)
    slots = i32([(pages - n) * PAGE + 5, pages * PAGE - 1])
    assert all(torch.equal(a, b) for a, b in zip(kv.read(cache, slots), kv.read(part, i32([5, n * PAGE - 1]))))
    q = dev(small.q.reshape(4, -1))
    x = torch.cat([q, torch.ones(4, 2 * hk * dim, dtype=torch.float16, device="cuda")], 1)
    last = i32([pages * PAGE - 4 + i for i in range(4)])
    cache.v_unit = torch.full((hk,), 0.125, device="cuda")
    kv.rope_append(cache, x, 16, i32([0] * 4), last, None)
    # 1 / (6 * 0.125) = 4/3 rounds to the scale 1.375; 1 / (1.375 / 8) = 5.8 to the code 6
    assert np.array_equal(host(kv.read(cache, last)[1]), np.full((4, hk * dim), 6 * 1.375 / 8))


@pytest.mark.parametrize("rows", [8, 70])
def test_attention_strides_scratch_streams(kv, rows):
    c = AttnCase4(kv, [(rows, 3000), (1, 200)], 10, 2, 128, 13)
    ref = c.run()
    c.check(ref)
    cache, n = c.device(), rows + 1
    row_start, seq, table = i32(c.row_start), i32(c.seq), i32(c.table)
    wide = torch.zeros(n, 10 * 128 + 40, dtype=torch.float16, device="cuda")
    q = wide[:, 16:16 + 1280]
    q[:] = dev(c.q.reshape(n, -1))
    out = torch.zeros(n, 1280 + 12, dtype=torch.float16, device="cuda")[:, 4:1284]
    tw = torch.full((2, c.width + 5), -1, dtype=torch.int32, device="cuda")
    tw[:, :c.width] = table
    kv.attention(cache, q, row_start, seq, tw[:, :c.width], rows, out=out)
    assert np.array_equal(host(out).reshape(ref.shape), ref)
    # any hint of the rows, any scratch: the same to rounding
    need = kv.attention4_scratch_bytes(2, rows, 10, 2, 128, c.width)
    for most in (0, 1, 3, 100):
        for size in (0, kv.SCRATCH_ZEROED, kv.SCRATCH_ZEROED + 30000, need // 2, need):
            s = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
            s[kv.SCRATCH_ZEROED:] = 255
            y = kv.attention(cache, q, row_start, seq, table, most, scratch_=s[:size] if size else s[:0])
            c.check(host(y).reshape(ref.shape).astype(np.float64))
            assert int(s[:kv.SCRATCH_ZEROED].count_nonzero()) == 0
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    ys = [kv.attention(cache, q, row_start, seq, table, rows, stream=s) for s in streams for _ in range(3)]
    for y in ys:
        assert np.array_equal(host(y).reshape(ref.shape), ref)


# ---------------------------------------------------------------- the set, as it is used

@pytest.mark.parametrize("dim,hq,hk,rows", [(128, 10, 2, 8), (64, 4, 4, 1), (256, 4, 1, 5), (128, 6, 2, 70)])
def test_a_round_from_a_graph(kv, dim, hq, hk, rows):
    # plan, append, attention, read back, log probabilities, eager and replayed: what a round leaves is what the
    # references give for what its cache holds
    rng = np.random.default_rng(21)
    before, vocab, pages = 300, 5000, 10
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def state():
        return dict(cache=kv.KvCache4.empty(pages, hk, dim), table=z(1, pages), free=torch.arange(pages, device="cuda").int(),
                    held=z(1), count=z(1) + pages, before=z(1))
    x = dev(rng.standard_normal((before + 4 * rows, (hq + 2 * hk) * dim)).astype(np.float16))
    logits = dev((3 * rng.standard_normal((rows, vocab))).astype(np.float16))
    tokens = i32(rng.integers(0, vocab, rows))
    f = dev((1e4 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32))
    w = dev((1 + 0.1 * rng.standard_normal(dim)).astype(np.float16))

    def step(s, part, n):
        r = kv.plan_round(s["before"], z(1) + n, s["held"], s["table"], s["free"], s["count"], capacity=n)
        s["held"].copy_(r.held)
        s["count"].copy_(r.free_count)
        s["before"] += n
        q = kv.rope_append(s["cache"], part, hq, r.positions, r.slots, f, w, w)
        y = kv.attention(s["cache"], q, r.row_start, r.seq_lens, s["table"], n)
        return (q, y, *kv.read(s["cache"], r.slots), *kv.logprobs(logits[:n], tokens[:n], 5, 0.7))
    with torch.cuda.stream(stream):
        s, t = state(), state()
        part = torch.empty(rows, x.shape[1], dtype=torch.float16, device="cuda")
        for u in (s, t):
            for a in range(0, before, 100):
                kv.rope_append(u["cache"], x[a:a + 1], hq, z(1), z(1) - 1, None)     # (a row without a slot)
            n, u["held"], u["count"] = 0, z(1), z(1) + pages
            while n < before:
                r = kv.plan_round(u["before"], z(1) + 100, u["held"], u["table"], u["free"], u["count"], capacity=100)
                kv.rope_append(u["cache"], x[n:n + 100], hq, r.positions, r.slots, f, w, w)
                u["held"].copy_(r.held)
                u["count"].copy_(r.free_count)
                u["before"] += 100
                n += 100
        part.copy_(x[before:before + rows])
        eager = [[o.clone() for o in step(s, part, rows)]]
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = step(t, part, rows)
    for i in range(3):
        with torch.cuda.stream(stream):
            part.copy_(x[before + i * rows:before + (i + 1) * rows])
            if i:
                eager.append([o.clone() for o in step(s, part, rows)])
            g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, eager[i]):
            assert torch.equal(a, b)
    # against the references, from the cache's own bytes
    total = before + 3 * rows
    codes, scales = host_cache(s["cache"])
    k, v = (kv4_ref.values(codes[j], scales[j], np.full(hk, 0.125)) for j in range(2))
    q, y = (host(o).astype(np.float64).reshape(rows, hq, dim) for o in eager[-1][:2])
    table = host(s["table"])
    ref, mag = kv_ref.attention(q, k, v, [0, rows], [total], table, dim ** -0.5, 0)
    tol = (2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -24 * (40 * dim + total)) * mag + total * 2.0 ** -25 * np.abs(v).max()
           + 2.0 ** -25)
    assert (np.abs(y - ref) <= tol).all()
    at = np.arange(total - rows, total)
    for got, want in zip(eager[-1][2:4], (k, v)):
        assert np.array_equal(host(got).astype(np.float64), want[table[0, at // PAGE], :, at % PAGE].reshape(rows, -1))


def test_calls_beside_each_other(kv):
    # attention and log probabilities whose sums pass through scratch: threads on one stream, other streams, graphs
    c = AttnCase4(kv, [(8, 5000), (3, 900)], 10, 2, 128, 17)
    ref = c.run()
    c.check(ref)
    cache, args = c.device(), (i32(c.row_start), i32(c.seq), i32(c.table), 8)
    q = dev(c.q.reshape(11, -1))
    rng = np.random.default_rng(18)
    z, tokens = dev((3 * rng.standard_normal((4, 100001))).astype(np.float16)), i32(rng.integers(0, 100001, 4))
    assert kv.attention4_scratch_bytes(2, 8, 10, 2, 128, c.width) > kv.SCRATCH_ZEROED
    assert kv.logprobs_scratch_bytes(4, 100001) > kv.SCRATCH_ZEROED
    want = [host(t) for t in (kv.attention(cache, q, *args), *kv.logprobs(z, tokens, 7))]
    torch.cuda.synchronize()

    def both(stream=None):
        return [kv.attention(cache, q, *args, stream=stream), *kv.logprobs(z, tokens, 7, stream=stream)]

    def same(got):
        for g, w in zip(got, want):
            assert np.array_equal(host(g), w)
    one, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(3)]
    got = [[] for _ in range(4)]

    def work(i):
        got[i] += [both(one) for _ in range(8)]
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(g) for g in got] == [8] * 4
    for g in got:
        for outs in g:
            same(outs)
    log("streams")
    outs = [both(s) for _ in range(4) for s in others]
    torch.cuda.synchronize()
    for o in outs:
        same(o)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=one):
            graphs.append((g, both() + both()))
    for rep in range(4):
        log(f"two graphs beside calls, {rep}")
        for _, out in graphs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, others):
            with torch.cuda.stream(s):
                g.replay()
        eager = both(one)
        torch.cuda.synchronize()
        for out in (eager, *(o[i:i + 5] for _, o in graphs for i in (0, 5))):
            same(out)


# ---------------------------------------------------------------- calls that a server makes and the above leave out

@pytest.mark.parametrize("rows", [3, 70])
def test_attention_queries_that_are_no_numbers(kv, rows):
    # a NaN query has no scores; an infinite one's are infinite, or NaN where the key's code is zero: NaN throughout the
    # row in either case, and nothing in the others
    c = AttnCase4(kv, [(rows, 100)], 4, 1, 64, 10)
    clean = c.run()
    c.q[1, 2, 5] = np.inf
    c.q[2, 0, 0] = np.nan
    c.q[0, 3, 63] = -np.inf
    y = c.run()
    hit = np.zeros(y.shape, bool)
    hit[1, 2] = hit[2, 0] = hit[0, 3] = True
    assert np.array_equal(np.isnan(y), hit)
    assert np.array_equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dim,hq,hk", [(128, 40, 8), (64, 40, 8), (256, 20, 4), (128, 10, 2)])
@pytest.mark.parametrize("width", [1024, 1025, 4096])
@pytest.mark.parametrize("lens", [[(8, 300)], [(8, 5001)], [(1, 700)], [(70, 900)], [(8, 200), (3, 900), (0, 70), (5, 64)]])
def test_attention_tables_wider_than_any_request(kv, dim, hq, hk, width, lens):
    # a server's tables are as wide as its longest context, and what lies behind a request's pages is anything; the
    # width decides whether the row tiles of a KV head are taken together
    c = AttnCase4(kv, lens, hq, hk, dim, 31)
    pages = c.codes.shape[1]
    wide = np.random.default_rng(4).choice([-7, 0, pages - 1, pages, 2 ** 31 - 1, -2 ** 31], (len(lens), width))
    wide[:, :c.width][c.table >= 0] = c.table[c.table >= 0]
    c.table = wide
    q = dev(c.q.reshape(c.q.shape[0], -1))
    for window in (0, 100):
        log(f"attention {lens} heads {hq}/{hk} dim {dim} table {width} window {window}")
        y = kv.attention(c.device(), q, i32(c.row_start), i32(c.seq), i32(c.table), max(r for r, _ in lens), window=window)
        c.table = np.clip(wide, 0, pages - 1)                      # (for the reference, which looks at what is seen alone)
        c.check(host(y).reshape(c.q.shape).astype(np.float64), window)
        c.table = wide


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_many_rows_far_offsets(kv, dim):
    # codes of over 2^32 bytes a side, a prompt block over the last pages, with a NaN group that its rows see in part
    pages, hk = 70000 * 256 // dim, 8
    small = AttnCase4(kv, [(150, 700)], 16, hk, dim, 12, extra_pages=0)
    n = small.codes.shape[1]
    small.scale[1, small.table[0, 9], 3, 20, 1] = 0x7F
    cache, part = kv.KvCache4.empty(pages, hk, dim), small.device()
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(cache, name).view(torch.uint8)[pages - n:] = getattr(part, name).view(torch.uint8)
    cache.k_unit, cache.v_unit = part.k_unit, part.v_unit
    clean = small.run()
    hit = np.zeros(clean.shape, bool)
    hit[9 * PAGE + 20 - 550:, 6:8, 16:32] = True                   # rows from the group's own token on
    assert np.array_equal(np.isnan(clean), hit)
    small.table = np.where(small.table >= 0, small.table + pages - n, small.table)
    assert np.array_equal(small.run(cache), clean, equal_nan=True)
