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
