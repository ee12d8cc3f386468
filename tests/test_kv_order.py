"""The order of FP16 logits that the log probabilities choose their likeliest tokens by (csrc/qpn_kv_order.h),
compiled for the host: every bit pattern.  No kernel is launched here."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_quantized_skinny_qpn_amd", "csrc")
SOURCE = """
#include "qpn_kv_order.h"
extern "C" {
uint32_t ordered_bits(uint32_t b) { return qpn::ordered_bits(b); }
uint32_t bits_of_ordered(uint32_t o) { return qpn::bits_of_ordered(o); }
uint64_t key_of(uint32_t o, uint32_t i) { return qpn::key_of(o, i); }
int index_of(uint64_t key) { return qpn::index_of(key); }
}
"""
BITS = np.arange(65536, dtype=np.uint16)
VALUES = BITS.view(np.float16).astype(np.float64)
NAN = np.isnan(VALUES)


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    at = tmp_path_factory.mktemp("order")
    (at / "order.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, str(at / "order.cpp"), "-o",
                    str(at / "order.so")], check=True)
    lib = ctypes.CDLL(str(at / "order.so"))
    lib.ordered_bits.restype = lib.bits_of_ordered.restype = ctypes.c_uint32
    lib.key_of.restype, lib.key_of.argtypes = ctypes.c_uint64, [ctypes.c_uint32] * 2
    lib.index_of.argtypes = [ctypes.c_uint64]
    return lib


def test_every_pattern_has_a_place(order):
    o = np.array([order.ordered_bits(int(b)) for b in BITS], np.int64)
    # 0 is what stands for no token: a list of tokens that count as none is never cut
    assert o.min() >= 1 and o.max() <= 0xFFFF
    v, p = VALUES[~NAN], o[~NAN]
    by = np.argsort(v, kind="stable")
    assert (np.sign(np.diff(p[by])) == np.sign(np.diff(v[by]))).all()      # the same order, and equal where they are
    back = np.array([order.bits_of_ordered(int(x)) for x in p], np.uint16).view(np.float16)
    assert np.array_equal(back.astype(np.float64), v)
    # NaN is never taken for a number
    assert not np.isin(o[NAN], p).any()


def test_keys(order):
    rng = np.random.default_rng(0)
    places = [int(x) for x in rng.integers(1, 65536, 200)] + [1, 0xFFFF]
    indices = [0, 1, 2 ** 24 - 1] + [int(x) for x in rng.integers(0, 2 ** 24, 20)]
    keys = [(order.key_of(o, i), o, i) for o in places for i in indices]
    assert all(k and k >> 32 == o and order.index_of(k) == i for k, o, i in keys)
    assert [(o, i) for _, o, i in sorted(keys, reverse=True)] == sorted(((o, i) for _, o, i in keys), key=lambda x: (-x[0], x[1]))
