"""Keys and values in one allocation: what the append refuses because a key's row and a value's would
share bytes, and which interleavings it takes (host-side checks, no GPU work)."""

import pytest

from activation_sparse_tiered_amd import _lib
from tests.test_layer_ops_abi import FAKE, _append, _cache, needs_no_gpu

PAGES, HEADS, ROWS, DIM = 8, 2, 16, 128     # _cache's, two bytes a value
ROW, HEAD, PAGE = DIM, ROWS * DIM, HEADS * ROWS * DIM


def _status(**kw):
    return _lib.lib.spax_kv_append(_append(_cache(**kw)), 0)


def _strides(page, head, row):
    return {f"{t}_{n}_stride": s for t in "kv" for n, s in (("page", page), ("head", head), ("row", row))}


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    dict(v=FAKE),
    dict(v=FAKE + 2 * ROW), dict(v=FAKE + 2 * HEAD), dict(v=FAKE + 2 * PAGE),
    dict(v=FAKE + 2 * 3 * PAGE), dict(v=FAKE + 2 * (PAGES - 1) * PAGE), dict(v=FAKE - 2 * ROW),
    dict(v=FAKE + 16),                                            # part of a row
    dict(v=FAKE + 2 * HEAD, **_strides(2 * PAGE, HEAD, ROW)),     # a page of k reaches v's
    dict(v=FAKE + 2 * ROW, **_strides(4 * HEAD, 2 * HEAD, ROW)),  # rows of a head are side by side
    # the same page, with its axes in another order
    dict(v=FAKE + 2 * PAGE, v_head_stride=DIM, v_row_stride=HEADS * DIM),
    dict(v=FAKE + 2 * PAGE, k_page_stride=2 * PAGE, v_page_stride=3 * PAGE),
], ids=str)
def test_shared_rows_are_refused(kw):
    assert _status(**kw) == _lib.SPAX_ERR_PARAM
    assert b"overlaps" in _lib.lib.spax_last_error()


@needs_no_gpu
@pytest.mark.parametrize("kw", [
    dict(v=FAKE + 2 * PAGES * PAGE), dict(v=FAKE - 2 * PAGES * PAGE),     # one after the other
    dict(v=FAKE + 2 * PAGE, **_strides(2 * PAGE, HEAD, ROW)),             # page by page
    dict(v=FAKE - 2 * PAGE, **_strides(2 * PAGE, HEAD, ROW)),
    dict(v=FAKE + 2 * PAGE, **_strides(5 * PAGE, HEAD, ROW)),
    dict(v=FAKE + 2 * HEAD, **_strides(2 * PAGE, 2 * HEAD, ROW)),         # head by head
    dict(v=FAKE + 2 * ROW, **_strides(2 * PAGE, 2 * HEAD, 2 * ROW)),      # row by row
    dict(v=FAKE + 2 * 2 * ROW, **_strides(2 * PAGE, ROW, 4 * ROW)),       # a token's heads together
    dict(v=FAKE + 2 * PAGES * HEAD, **_strides(HEAD, 2 * PAGES * HEAD, ROW)),   # heads outermost
    # a page's halves, each with its own order of axes
    dict(v=FAKE + 2 * PAGE, k_page_stride=2 * PAGE, v_page_stride=2 * PAGE, v_head_stride=DIM,
         v_row_stride=HEADS * DIM),
], ids=str)
def test_interleavings_without_a_shared_row_reach_the_launch(kw):
    # every check passed: what fails is the launch, without a device
    assert _status(**kw) == _lib.SPAX_ERR_HIP, _lib.lib.spax_last_error()
