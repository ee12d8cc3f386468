"""GPU parity of the log probabilities against the plain FP64 reference (kv4_ref.logprobs).

Tolerances, derived before the first run.  Of a row with x = (z - max) / T: the exponentials are off by
2^-23 (1 + |x|) of themselves (argument and result in FP32, a factor 2 for the hardware's), and those that
make up all but 2^-40 of the sum have |x| < 28 + log n < 45: S - 1 is off by 46 * 2^-22 of itself, log S by
d = 46 * 2^-22 min(S - 1, 1) at most, the entropy by as much, and by as much again of itself for its own sum
of x exp(x); results are rounded to FP32 (2^-24).  Ids are equal.
"""
import numpy as np
import pytest
import torch

import kv4_ref
from gpu_util import dev, host, log, need_gpu
from test_gpu_kv import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv():
    need_gpu()
    from fp8_quantized_skinny_qpn_amd import kv as k
    return k


def check(kv, z, tokens, top, temperature=1.0, zd=None, **more):
    rows, n = z.shape
    log(f"logprobs {rows} x {n} top {top}")
    zd = dev(z) if zd is None else zd
    torch.cuda.synchronize()
    got = kv.logprobs(zd, i32(tokens), top, temperature, **more)
    lp, h, ids, lps = (host(t).astype(np.float64) for t in got)
    with np.errstate(all="ignore"):
        rl, rh, rids, rlps = kv4_ref.logprobs(z, tokens, top, 1.0 / temperature)
        best = z.astype(np.float64).max(1, keepdims=True)
        s1 = np.exp((z.astype(np.float64) - best) / temperature).sum(1) - 1
    assert np.array_equal(ids, rids)
    d = 46 * 2.0 ** -22 * np.minimum(np.maximum(s1, 0), 1) + 2.0 ** -50
    for a, b, e in ((lp, rl, d), (h, rh, d + 46 * 2.0 ** -22 * np.abs(rh)), (lps, rlps, d[:, None])):
        # FP32 rounds what is 2^128 - 2^103 or more (its largest number and half a step) to infinity
        b = np.where(np.abs(b) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(np.inf, b), b)
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
        ok = np.isfinite(b)
        assert np.array_equal(a[np.isinf(b)], b[np.isinf(b)])
        with np.errstate(invalid="ignore"):
            err, tol = np.abs(a - b), 2.0 ** -24 * np.abs(b) + e
        assert (err <= tol)[ok].all(), f"{(err / tol)[ok].max():.2f} of what is allowed"
    return got


@pytest.mark.parametrize("rows,n", [(1, 1), (1, 2), (3, 7), (2, 8), (1, 1000), (5, 4095), (2, 4097), (8, 5001), (1, 50000),
                                    (8, 151936), (1, 151936), (40, 20001), (300, 1500), (1100, 1030), (1030, 9000)])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 32])
def test_logprobs(kv, rows, n, top):
    rng = np.random.default_rng(rows + n)
    z = (3 * rng.standard_normal((rows, n))).astype(np.float16)
    tokens = rng.integers(0, n, rows)
    tokens[0] = z[0].argmax()
    check(kv, z, tokens, min(top, n), 0.8)


@pytest.mark.parametrize("temperature", [1e-3, 0.3, 1.0, 7.0, 1e4])
def test_temperatures(kv, temperature):
    rng = np.random.default_rng(2)
    z = (4 * rng.standard_normal((6, 3001))).astype(np.float16)
    check(kv, z, z.argsort(1)[:, -2], 20, temperature)


@pytest.mark.parametrize("temperature", [1e10, 1e40, 1e300, 1e-10, 1e-40])
def test_far_temperatures_with_masked_tokens(kv, temperature):
    rng = np.random.default_rng(9)
    z = (3 * rng.standard_normal((4, 3000))).astype(np.float16)
    z[:, ::3] = -np.inf
    z[1, :2990] = -np.inf
    z[2] = np.float16(65504) * rng.choice([-1, 1], 3000)
    check(kv, z, [1, 2995, 5, 0], 8, temperature)


def test_likely_tokens_keep_their_precision(kv):
    # one token takes all but 1e-3 .. 1e-9: its log probability is that difference, not 0
    rng = np.random.default_rng(3)
    z = rng.standard_normal((12, 30000)).astype(np.float16)
    at = rng.integers(0, 30000, 12)
    z[np.arange(12), at] = 18 + 1.25 * np.arange(12)
    lp = host(check(kv, z, at, 4)[0])
    assert (lp < 0).all() and lp[-1] > -1e-8


def test_ties_go_to_the_lowest_index(kv):
    rng = np.random.default_rng(4)
    z = rng.integers(-3, 4, (9, 20011)).astype(np.float16)      # thousands of equal ones
    z[1] = 0.0                                                  # all equal
    z[2] = np.where(rng.random(20011) < 0.5, -0.0, 0.0)         # -0 and 0 are
    z[3] = -np.inf
    z[3, [17, 20010, 5000]] = [1.0, 1.0, 0.5]                   # three with any probability
    z[4] = np.arange(20011) // 700                              # rising, in steps
    z[5] = -(np.arange(20011) // 700)
    z[6] = -np.inf
    z[6, 20010] = -65504.0
    z[7] = 65504.0
    z[8] = -65504.0
    for top in (1, 20, 32):
        check(kv, z, rng.integers(0, 20011, 9), top)


def test_bad_rows_and_tokens(kv):
    rng = np.random.default_rng(5)
    z = rng.standard_normal((10, 9001)).astype(np.float16)
    z[1, 5000] = np.nan
    z[2, 0] = np.inf
    z[3] = -np.inf
    z[4] = np.nan
    z[5, 100:] = -np.inf
    z[6, 9000] = np.inf
    z[6, 3] = -np.inf
    tokens = np.array([-1, 0, 0, 0, 0, 200, 9000, 9001, 2 ** 31 - 1, -2 ** 31])
    for top in (0, 20):
        check(kv, z, tokens, top)


def test_strides_alignments_and_streams(kv):
    rng = np.random.default_rng(6)
    n = 8193
    z = (2 * rng.standard_normal((7, n))).astype(np.float16)
    tokens = rng.integers(0, n, 7)
    want = [host(t) for t in check(kv, z, tokens, 9)]
    for stride, offset in ((n, 0), (n + 7, 3), (n + 1, 1), (n + 15, 7), (n + 8, 8)):
        flat = torch.full((7 * stride + 64,), float("nan"), dtype=torch.float16, device="cuda")
        wide = flat[offset:offset + 7 * stride].view(7, stride)[:, :n]
        wide.copy_(dev(z))
        got = check(kv, z, tokens, 9, zd=wide, stream=torch.cuda.Stream())
        for a, b in zip(got, want):            # the same tokens in other lanes: the sums' order may differ
            assert np.allclose(host(a), b, rtol=2e-6, atol=1e-9)


def test_scratch_outputs_and_graphs(kv):
    rng = np.random.default_rng(7)
    n = 60001
    zs = [dev((2 * rng.standard_normal((4, n))).astype(np.float16)) for _ in range(3)]
    tokens = i32(rng.integers(0, n, 4))
    want = [[host(t).copy() for t in kv.logprobs(z, tokens, 20)] for z in zs]
    need = kv.logprobs_scratch_bytes(4, n)
    s = torch.zeros(need, dtype=torch.uint8, device="cuda")
    s[kv.SCRATCH_ZEROED:] = 255
    for z, w in zip(zs, want):
        assert all(np.array_equal(host(a), b) for a, b in zip(kv.logprobs(z, tokens, 20, scratch_=s), w))
        assert int(s[:kv.SCRATCH_ZEROED].count_nonzero()) == 0
    out = (torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, 20, dtype=torch.int32, device="cuda"),
           torch.empty(4, 20, device="cuda"))
    z = torch.empty_like(zs[0])
    stream, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        kv.logprobs(z, tokens, 20, out=out)
        again = kv.logprobs(z, tokens, 20)
    for i in range(4):
        z.copy_(zs[i % 3])
        eager = kv.logprobs(zs[(i + 1) % 3], tokens, 20)
        g.replay()
        torch.cuda.synchronize()
        for got, w in ((out, want[i % 3]), (again, want[i % 3]), (eager, want[(i + 1) % 3])):
            assert all(np.array_equal(host(a), b) for a, b in zip(got, w))


@pytest.mark.parametrize("n,rows", [(700, 9), (5000, 9), (40001, 9), (40001, 300)])   # a tile, a piece, several pieces, one
@pytest.mark.parametrize("bits", [0xFFFF, 0xFFFE, 0xFE00, 0xFC01, 0x7FFF, 0x7E00, 0x7C01])
def test_nan_of_any_bits(kv, n, rows, bits):
    # whole rows, tiles, the ends of rows and single tokens of it, among numbers and among masked ones; every other row
    # holds numbers alone
    rng = np.random.default_rng(n)
    z = (3 * rng.standard_normal((rows, n))).astype(np.float16)
    u = z.view(np.uint16)
    u[1] = bits
    u[3, n // 2:n // 2 + 1024] = bits
    u[5] = 0xFC00
    u[5, ::2] = bits
    u[7] = 0xFC00
    u[7, [0, n - 1]] = 0x3C00, bits
    z[8, 3:] = -np.inf
    if rows > 100:
        u[100:164:2, ::3] = bits
    tokens = rng.integers(0, n, rows)
    for top in (0, 1, 20, 32):
        check(kv, z, tokens, top)


@pytest.mark.parametrize("rows,n", [(1, 151936), (9, 20011), (300, 9001)])
def test_rows_of_few_values(kv, rows, n):
    # what a grammar leaves: fewer tokens than are asked for, the rest masked; and rows of a few different values
    rng = np.random.default_rng(rows)
    z = np.full((rows, n), -np.inf, np.float16)
    for r in range(rows):
        if r % 3 == 2:
            z[r] = rng.integers(-1, 2, n)
        else:
            at = rng.choice(n, 3 + 30 * (r % 3), replace=False)
            z[r, at] = rng.standard_normal(len(at))
    for top in (1, 20, 32):
        check(kv, z, rng.integers(0, n, rows), top)


def test_far_rows(kv):
    # rows more than 2^32 bytes behind the first
    rows, n, stride = 2060, 1000, 1 << 20
    rng = np.random.default_rng(8)
    z = (3 * rng.standard_normal((rows, n))).astype(np.float16)
    flat = torch.empty(rows * stride, dtype=torch.float16, device="cuda")
    wide = flat.view(rows, stride)[:, :n]
    wide.copy_(dev(z))
    assert (rows - 1) * stride * 2 > 2 ** 32
    check(kv, z, rng.integers(0, n, rows), 5, zd=wide)
