"""The speculative-round operators at the edges of what they accept.

References and tolerances are those of test_gpu_kv.py; where one differs it is derived at its test.
"""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_kv import PAGE, AttnCase

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
