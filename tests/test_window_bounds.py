"""Bounds of attn_fwd_window's host side (no GPU)."""

import ctypes

import numpy as np

from tests.test_window_plan import rkv  # noqa: F401


def test_plan_refuses_more_units_than_items_number(rkv):  # noqa: F811
    """A work item's number has 30 bits: the plan refuses what the launch refuses.  2^20 heads of 524,288 rows
    in units of 512 are 2^30 units (no unit_tiles: the refusal comes before they are written)."""
    Lq, H = 512 * 1024, 1 << 20
    s, w, rope = rkv.rkv_attn_seq(Lq=Lq, Lk=10, block_frames=1), rkv.rkv_attn_window(3, 0), rkv.make_rope(1, 1)
    rows = [np.zeros(Lq, dtype=np.int64) for _ in range(3)]
    n = ctypes.c_int64(-1)

    def plan(heads):
        return rkv.lib().rkv_attn_window_rows(ctypes.byref(s), ctypes.byref(w), 1, heads, heads, ctypes.byref(rope),
                                              *[r.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)) for r in rows], None,
                                              ctypes.byref(n))

    assert plan(H) == rkv.RKV_ERR_UNSUPPORTED
    assert "units" in rkv.rkv_last_error_string() and n.value == -1
    assert plan(H - 1) == rkv.RKV_OK and n.value == (H - 1) * 1024
