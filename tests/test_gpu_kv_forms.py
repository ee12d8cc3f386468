"""The speculative-round operators where their kernels change form: many query rows, joins of many
pieces, long vocabularies, rotations of every width, scratch under capture, rows that requests share.

References and tolerances are those of test_gpu_kv.py (derived there from the roundings that the
kernels make); results that a change must not touch are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import kv_ref
from gpu_util import dev, host, log, need_gpu
from test_gpu_kv import PAGE, AttnCase, append_case, check_plan, check_verify, i32, run_slots, verify_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    need_gpu()
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


# ---------------------------------------------------------------- attention, many rows

# rows of a KV head: 60 x 5 and 40 x 1 cross the forms at 48, 17 x 5 = 85 and 30 x 4 = 120 need up to 8 tiles
MANY = [(60, 300), (1, 1), (0, 500), (33, 33), (60, 64), (5, 1300), (1, 129), (0, 0), (50, 1500), (40, 70)]


@pytest.mark.parametrize("dim,hq,hk", [(128, 10, 2), (64, 4, 4), (64, 4, 2), (256, 8, 1), (128, 4, 2)])
@pytest.mark.parametrize("window", [0, 1, 70, 1000])
def test_attention_many_rows_ragged_and_windows(kv, dim, hq, hk, window):
    c = AttnCase(kv, MANY, hq, hk, dim, 31)
    c.check(c.run(window=window), window)


@pytest.mark.parametrize("dim,hq,hk", [(128, 5, 1), (64, 8, 4), (256, 2, 1), (128, 1, 1)])
@pytest.mark.parametrize("rows", [9, 10, 17, 25, 48, 49, 129])
def test_attention_every_tile_count(kv, dim, hq, hk, rows):
    c = AttnCase(kv, [(rows, rows + 131)], hq, hk, dim, 32 + rows)
    c.check(c.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_many_rows_unseen_tokens_never_matter(kv, dim, window):
    c = AttnCase(kv, [(70, 150), (50, 64), (60, 321)], 4, 2, dim, 33)
    clean = c.run(window=window)
    c.check(clean, window)
    used = np.zeros(c.codes.shape[1:4], bool)
    for r, (n, t) in enumerate(c.lens):
        for j in range(max(0, t - n + 1 - window) if window else 0, t):
            used[c.table[r, j // PAGE], :, j % PAGE] = True
    for junk in (0x7F, 0xFF, 0x7E):
        codes = c.codes.copy()
        c.codes[:, ~used] = junk
        assert np.array_equal(c.run(window=window), clean), hex(junk)
        c.codes = codes
    # request 0, KV head 1: a value of position 100 (row 20 of 70), dimension 17
    p, last = 100, 70 if not window else 20 + window
    c.codes[1, c.table[0, p // PAGE], 1, p % PAGE, 17] = 0x7F
    hit = np.zeros(clean.shape, bool)
    hit[20:min(last, 70), 2:4, 17] = True
    y = c.run(window=window)
    assert np.array_equal(np.isnan(y), hit) and np.array_equal(y[~hit], clean[~hit])
    c.codes[0, c.table[0, p // PAGE], 1, p % PAGE, 3] = 0xFF
    hit[20:min(last, 70), 2:4, :] = True
    y = c.run(window=window)
    assert np.array_equal(np.isnan(y), hit) and np.array_equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_many_rows_bad_pages_and_lengths(kv, dim):
    c = AttnCase(kv, [(60, 200), (70, 200), (50, 90)], 4, 2, dim, 34)
    clean = c.run()
    mine = slice(60, 130)
    others = np.r_[0:60, 130:180]
    for bad in (-1, c.codes.shape[1], 2 ** 31 - 1, -2 ** 31):
        keep = c.table.copy()
        c.table[1, 1] = bad                  # tokens 64 .. 127; the request's rows stand at 130 .. 199
        y = c.run()
        assert np.isnan(y[mine]).all() and np.array_equal(y[others], clean[others])
        y = c.run(window=3)                  # rows at 130 and behind see nothing before 128
        assert np.isfinite(y).all()
        c.table = keep
    c.seq = [200, 64 * c.width + 1, 90]
    y = c.run()
    assert np.isnan(y[mine]).all() and np.array_equal(y[others], clean[others])
    c.seq = [200, 0, -5]
    y = c.run()
    assert np.array_equal(y[:60], clean[:60]) and not y[60:].any()


@pytest.mark.parametrize("rows,hq,hk", [(8, 10, 2), (60, 10, 2), (60, 2, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_scales_out_of_proportion(kv, rows, hq, hk, dim):
    if dim == 256 and hq == 10:
        hq = 8
    c = AttnCase(kv, [(rows, 1500)], hq, hk, dim, 35)
    c.scale[1] *= 2.0 ** np.random.default_rng(1).integers(-45, 1, c.scale[1].shape)   # from page to page
    c.check(c.run())
    c.scale[1, ::3] = 0.0                                     # pages of zeros among others
    c.check(c.run())
    c.scale[1] = 0.0
    assert not c.run().any()
    c.scale[1] = 1.5                                          # no power of two
    c.scale[0] *= 0.7
    c.check(c.run())
    c.scale[0] = 0.0
    c.check(c.run())                                          # all scores equal
    c.scale[1, c.table[0, 1], 0] = -1.0                       # not a scale: NaN, not a wrong number
    y = c.run()
    assert np.isnan(y[:, :hq // hk]).all() and np.isfinite(y[:, hq // hk:]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_many_rows_peaked_scores(kv, dim):
    # scores up to some +-40: the running maximum is raised again and again
    c = AttnCase(kv, [(64, 1500)], 10, 2, dim, 36, size=8.0)
    c.check(c.run())


@pytest.mark.parametrize("rows,hq,dim", [(1, 1, 64), (8, 5, 128), (2, 8, 256), (64, 2, 128), (40, 4, 64), (20, 4, 256)])
def test_attention_joins_of_many_pieces(kv, rows, hq, dim):
    # one KV head of a long cache: more pieces than one step joins, the last one short
    c = AttnCase(kv, [(rows, 64 * 200 + 7)], hq, 1, dim, 37)
    c.check(c.run())


def test_attention_many_rows_any_hint_and_scratch(kv):
    c = AttnCase(kv, [(60, 1700), (1, 200), (9, 900)], 10, 2, 128, 38)
    q, row_start, seq, table = dev(c.q.reshape(70, -1)), i32(c.row_start), i32(c.seq), i32(c.table)
    cache = c.device()
    need = kv.attention_scratch_bytes(3, 60, 10, 2, 128, c.width)
    for most in (0, 1, 5, 10, 60, 5000):
        for size in (0, kv.SCRATCH_ZEROED, kv.SCRATCH_ZEROED + 200000, need):
            log(f"hint {most} scratch {size}")
            s = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
            s[kv.SCRATCH_ZEROED:] = 255
            y = kv.attention(cache, q, row_start, seq, table, most, scratch_=s[:size])
            c.check(host(y).reshape(c.q.shape).astype(np.float64))
            assert int(s[:kv.SCRATCH_ZEROED].count_nonzero()) == 0


@pytest.mark.parametrize("dim", [64, 256])
def test_attention_many_rows_infinite_queries(kv, dim):
    c = AttnCase(kv, [(60, 100)], 4, 1, dim, 39)
    clean = c.run()
    c.q[1, 2, 5] = np.inf
    c.q[50, 0, 0] = np.nan
    y = c.run()
    hit = np.zeros(y.shape, bool)
    hit[1, 2] = hit[50, 0] = True
    assert np.isnan(y[hit]).all() and np.array_equal(y[~hit], clean[~hit])


def test_attention_rows_of_two_requests(kv):
    # rows that two requests name belong to either; the other rows to theirs
    c = AttnCase(kv, [(4, 300), (0, 0), (8, 700)], 4, 2, 64, 40)
    first = AttnCase.run(c)
    c.row_start = np.array([0, 4, 0, 8])
    q = dev(c.q.reshape(12, -1))
    y = host(kv.attention(c.device(), q, i32(c.row_start), i32(c.seq), i32(c.table), 8)).reshape(c.q.shape)
    k, v = c.values()
    table = np.clip(c.table, 0, None)
    ref, mag = kv_ref.attention(c.q[:8].astype(np.float64), k, v, [0, 8], c.seq[2:], table[2:], 64 ** -0.5, 0)
    tol = 2.0 ** -11 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -24 * (40 * 64 + 700)) * mag + 700 * 2.0 ** -25 * np.abs(v).max() + 2.0 ** -25
    assert (np.abs(y[4:8] - ref[4:]) <= tol[4:]).all()
    own = (np.abs(y[:4] - ref[:4]) <= tol[:4]).all((1, 2))
    assert (own | (y[:4] == first[:4]).all((1, 2))).all()


def test_scratch_made_under_capture_is_the_graphs_own(kv):
    c = AttnCase(kv, [(8, 3000)], 10, 2, 128, 41)
    want = c.run()
    q, row_start, seq, table, cache = dev(c.q.reshape(8, -1)), i32(c.row_start), i32(c.seq), i32(c.table), c.device()
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    held = dict(kv._scratches)
    with torch.cuda.graph(graph, stream=side):
        kv.attention(cache, q, row_start, seq, table, 8, out=out)
    for key, s in kv._scratches.items():
        assert key in held and held[key] is s
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out).reshape(want.shape), want)
        assert np.array_equal(c.run(), want)


# ---------------------------------------------------------------- rope_append

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("part", [16, 48, -16, 0])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_rotation_widths(kv, dim, part, interleaved):
    rot = part if part > 0 else dim + part
    slots, pos = run_slots([(60, 9), (700, 2)], 6, dim)
    append_case(kv, dim, 6, 2, slots, pos, 6, dim + rot, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("dim,hq,hk", [(64, 12, 4), (128, 40, 8), (256, 4, 2)])
def test_append_prompt_blocks(kv, dim, hq, hk):
    # pages begun before, whole and ended inside, of several requests one after another
    slots, pos = run_slots([(1000, 300), (0, 130), (63, 66)], 14, dim)
    append_case(kv, dim, hq, hk, slots, pos, 14, 50 + dim)


def test_append_far_positions(kv):
    slots, _ = run_slots([(5, 6)], 2, 1)
    append_case(kv, 128, 4, 2, slots, [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 1, 10 ** 9, 2 ** 24 + 1, 0], 2, 60)


def test_append_one_row_a_page_in_falling_order(kv):
    # every row on its own page, pages descending; then all rows on one slot
    append_case(kv, 64, 2, 1, [p * PAGE + 63 - p for p in range(39, -1, -1)], list(range(40)), 40, 61)
    append_case(kv, 64, 2, 1, [70] * 40, list(range(40)), 3, 62)


# ---------------------------------------------------------------- verify_sampled

def accept_all(logits, draft, tokens, u, su):
    u[:] = 0.0


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("n", [4097, 300000])
def test_verify_many_rows_a_request(kv, n, sampled):
    # more rows than a workgroup holds the masses of, stopping behind them; more chunks than one step takes
    counts = [24, 3] if n < 10000 else [18, 1]

    def late(logits, draft, tokens, u, su):
        u[:] = 0.0
        u[20 if n < 10000 else 16] = 1.0
    for edit in (accept_all, late, None):
        got, ref, _ = verify_case(kv, counts, n, 70, sampled, edit=edit)
        check_verify(got, ref)


@pytest.mark.parametrize("sampled", [False, True])
def test_verify_long_vocabulary_one_row(kv, sampled):
    got, ref, _ = verify_case(kv, [2], 1 << 20, 71, sampled)
    check_verify(got, ref)


def test_verify_rows_of_two_requests(kv):
    got, ref, args = verify_case(kv, [4, 0, 8], 5000, 72, True)
    check_verify(got, ref)
    a = list(args)
    a[2] = i32([0, 4, 0, 8])                 # requests 0 and 2 share rows 0 .. 3
    got = [host(g) for g in kv.verify_sampled(*a)]
    logits, draft, tokens = host(a[0]), host(a[5]), host(a[1])
    u, su = host(a[3]), host(a[4])
    for r, (lo, hi) in ((0, (0, 4)), (2, (0, 8))):
        ref = kv_ref.verify(logits[lo:hi], draft[lo:hi], tokens[lo:hi], [0, hi - lo], 1 / 0.8, u[lo:hi], su[r:r + 1])
        assert got[0][r] == ref[0][0] and got[1][r] == ref[1][0]
    assert got[0][1] == 0 and got[1][1] == -1


def test_verify_rows_of_unlike_alignment(kv):
    # target and drafter rows that begin at different places of a 16-byte granule
    n, rows = 4999, 5
    got, ref, args = verify_case(kv, [3, 2], n, 73, True)
    check_verify(got, ref)
    for lead in range(1, 8):
        wide = torch.full((rows, n + 9), 9.0, dtype=torch.float16, device="cuda")
        part = wide[:, lead:lead + n]
        part.copy_(args[5])
        again = kv.verify_sampled(args[0], *args[1:5], part, 0.8)
        torch.cuda.synchronize()
        assert [host(g).tolist() for g in again[:2]] == [g.tolist() for g in got[:2]]
        check_verify([host(g) for g in again], ref)


# ---------------------------------------------------------------- plan_round

def test_plan_round_most_requests(kv):
    n = 4096
    before, rows = np.arange(n) * 7 % 300, np.arange(n) % 3
    held = -(-before // PAGE)
    width = 6
    free = np.random.default_rng(80).permutation(20000)
    check_plan(kv, before, rows, held, np.zeros((n, width), int), free, 20000, int(rows.sum()) + 100)
    check_plan(kv, before, rows, held, np.zeros((n, width), int), free, 500, 3000)


def test_plan_round_one_long_prompt(kv):
    check_plan(kv, [10, 64, 0], [100000, 0, 1], [1, 1, 0], np.zeros((3, 1600), int), list(range(1599, -1, -1)), 1600, 100001)
    check_plan(kv, [10, 64, 0], [100000, 0, 1], [1, 1, 0], np.zeros((3, 1600), int), list(range(1599, -1, -1)), 1600, 100000)
