"""Layouts the Python calls take and refuse, without a GPU: a tensor's stride
over a dimension of one says nothing."""

import pytest
import torch


@pytest.fixture(scope="module")
def rkv(lib_path):
    from rolling_kv_cache_rope_b200 import rkv as m
    return m


def test_row_stride_of_single_rows_and_heads(rkv):
    base = torch.zeros(8, 6, 128, dtype=torch.bfloat16)
    heads_first = torch.zeros(6, 1, 128, dtype=torch.bfloat16).transpose(0, 1)     # one token: contiguous
    one_head = torch.zeros(1, 9, 128, dtype=torch.bfloat16).transpose(0, 1)
    for t, want in ((base, 768), (base[:, :4], 768), (base[::2], 1536), (base[:1], 768), (base[2:3, 1:5], 512),
                    (base[:, 3:4], 768), (heads_first, 768), (one_head, 128)):
        got = rkv._row_stride(t, "x", t.shape, -1)
        assert got == want, (t.shape, t.stride(), got)
        for i in range(t.shape[0]):          # the stride leads from row to row
            assert t[i].data_ptr() == t.data_ptr() + 2 * got * i
    for t in (base.transpose(1, 2), base.transpose(0, 1), base[:, ::2], base[:, :1].transpose(0, 1)):
        with pytest.raises(ValueError):
            rkv._row_stride(t, "x", t.shape, -1)


def test_empty_page_tables(rkv):
    for shape in ((0, 4), (4, 0)):
        k = torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="page_table"):
            rkv._check_table(torch.zeros(shape, dtype=torch.int32), k.device)


def test_page_table_layouts(rkv):
    t = torch.zeros(6, 8, dtype=torch.int32)
    dev = t.device
    assert rkv._check_table(t, dev) == 8 and rkv._check_table(t[:, :5], dev) == 8 and rkv._check_table(t[::2], dev) == 16
    assert rkv._check_table(t[:1, :3], dev) == 3                       # one sequence: any stride will do
    assert rkv._check_table(torch.zeros(1, 6, dtype=torch.int32).t(), dev) == 1   # one page a sequence, stride 6 over it
    for bad in (t.t(), t[:, ::2], t.long(), t[0]):
        with pytest.raises(ValueError, match="page_table"):
            rkv._check_table(bad, dev)
