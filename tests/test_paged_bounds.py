"""What the paged calls refuse before a kernel runs: strides whose products pass
64 bits, and tensors that share bytes with what a call writes (no GPU)."""

import pytest

from tests.test_paged_abi import cache, decode, evict, insert, rkv  # noqa: F401


@pytest.mark.parametrize("call", [insert, decode, evict])
def test_table_strides_past_64_bits(rkv, call):  # noqa: F811
    assert call(rkv, cache(rkv, table_stride=1 << 61)) == rkv.RKV_ERR_INVALID_ARG
    assert "table_stride" in rkv.rkv_last_error_string()
    assert call(rkv, cache(rkv, table_stride=(1 << 32) + 1)) == rkv.RKV_ERR_INVALID_ARG
    # one sequence: its stride says nothing (the call gets as far as a workspace or an argument that is not there)
    one = dict(lens=0)
    assert call(rkv, cache(rkv, n_seqs=1, table_stride=1 << 61), **one) == rkv.RKV_ERR_INVALID_ARG
    assert "NULL" in rkv.rkv_last_error_string()


def test_row_strides_past_64_bits(rkv):  # noqa: F811
    many = dict(n_seqs=1 << 25, H=2, max_pages=1, table_stride=1, page_tokens=1, page_stride=256, n_pages=4)
    for kw in (dict(qs=1 << 39), dict(os=1 << 39)):
        assert decode(rkv, cache(rkv, **many), **kw) == rkv.RKV_ERR_INVALID_ARG
        assert "stride" in rkv.rkv_last_error_string()
    assert insert(rkv, cache(rkv, **many), stride=1 << 39) == rkv.RKV_ERR_INVALID_ARG
    assert "stride" in rkv.rkv_last_error_string()


# calls as they stand in test_paged_abi: k 0x1.., v 0x2.., table 0x3.., status 0x31.., q / k_new 0x40.., o / v_new 0x41..,
# seq_lens 0x50.., ws 0x60..
@pytest.mark.parametrize("change", [
    dict(win=0x410000000, wout=0x700000000),                     # o over what the weights are read from
    dict(win=0x410000000 - 4 * 2 * 128 * 4 + 4, wout=0x700000000),
    dict(o=0x300000000), dict(o=0x310000000 - 16), dict(wout=0x300000000), dict(wout=0x310000000),
    dict(ws=0x400000000), dict(ws=0x410000000), dict(ws=0x100000000), dict(ws=0x200000000 - 16), dict(ws=0x500000000 - 16),
    dict(ws=0x300000000), dict(ws=0x310000000 - 16), dict(ws=0x700000000, wout=0x700000000),
    dict(ws=0x700000000, win=0x700000000, wout=0x720000000),
    dict(q=0x310000000 - 16), dict(lens=0x310000000),
])
def test_decode_outputs_stand_apart(rkv, change):  # noqa: F811
    assert decode(rkv, cache(rkv), **change) == rkv.RKV_ERR_INVALID_ARG
    assert "overlap" in rkv.rkv_last_error_string()


@pytest.mark.parametrize("change", [
    dict(ws=0x500000000 - 16), dict(ws=0x510000000), dict(ws=0x520000000 - 16), dict(ws=0x530000000), dict(ws=0x100000000),
    dict(ws=0x300000000), dict(ws=0x310000000 - 16), dict(wout=0x700000000, pout=0x710000000, ws=0x710000000),
    dict(lens_out=0x700000000, ws=0x700000000), dict(wout=0x300000000, pout=0x720000000),
    dict(lens_out=0x300000000), dict(lens_out=0x310000000), dict(wout=0x720000000, pout=0x310000000),
    # out of place, scores and lengths that are only read, in the pool the call writes
    dict(weight=0x100000000, wout=0x700000000, pout=0x710000000), dict(pos=0x200000000, wout=0x700000000, pout=0x710000000),
    dict(nxt=0x100000000), dict(lens=0x100000000, lens_out=0x700000000),
])
def test_evict_outputs_stand_apart(rkv, change):  # noqa: F811
    assert evict(rkv, cache(rkv), **change) == rkv.RKV_ERR_INVALID_ARG
    assert "overlap" in rkv.rkv_last_error_string()


@pytest.mark.parametrize("change", [
    dict(lens=0x100000000), dict(nxt=0x200000000, pos=0x710000000), dict(weight=0x300000000), dict(weight=0x310000000),
    dict(nxt=0x700000000, pos=0x300000000), dict(k=0x310000000 - 16),
])
def test_insert_outputs_stand_apart(rkv, change):  # noqa: F811
    assert insert(rkv, cache(rkv), **change) == rkv.RKV_ERR_INVALID_ARG
    assert "overlap" in rkv.rkv_last_error_string()


@pytest.mark.parametrize("call", [insert, decode, evict])
@pytest.mark.parametrize("change", [dict(page_table=0x100000000), dict(status=0x200000000), dict(status=0x300000004)])
def test_table_and_status_stand_apart(rkv, call, change):  # noqa: F811
    if call is decode and "page_table" in change:
        return          # it writes neither
    assert call(rkv, cache(rkv, **change)) == rkv.RKV_ERR_INVALID_ARG
    assert "overlap" in rkv.rkv_last_error_string()


def test_neighbours_are_no_overlap(rkv):  # noqa: F811
    """Tensors that share a buffer without sharing bytes pass: the calls get as far as the workspace that is not there."""
    half = 16 * 2 * 128
    # pages of K and V and room between them; a table with room between its rows, the status word there
    c = cache(rkv, page_stride=8 * half, v=0x100000000 + 2 * half, table_stride=40, status=0x300000000 + 8 * 4)
    gap = 0x100000000 + 4 * half
    for call, kw in ((decode, dict(o=gap)), (decode, dict(q=0x400000000, o=0x400000000 + 1024, qs=1024, os=1024)),
                     (decode, dict(lens=0x300000000 + 20 * 4)), (decode, dict(win=0x700000000, wout=0x700000000)),
                     (evict, dict(lens=gap, lens_out=gap)), (evict, dict(lens_out=0x300000000 + 20 * 4)),
                     (evict, dict(wout=0x700000000, pout=0x710000000)), (evict, dict(nxt=gap))):
        assert call(rkv, c, ws=0, **kw) == rkv.RKV_ERR_INVALID_ARG
        assert "workspace must" in rkv.rkv_last_error_string(), (call, kw)
