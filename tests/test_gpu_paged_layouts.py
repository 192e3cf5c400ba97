"""Tensors of one token, one head, one page: their strides over a dimension of
one are whatever they are."""

import math

import pytest
import torch

from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import need_gpu, to_dev
from tests._paged import D, Streams, check_decode

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


def heads_first(t):
    """The same [1, H, D] tensor as a view of [H, 1, D]: contiguous, with strides (D, D, 1)."""
    out = t.reshape(t.shape[1], 1, t.shape[2]).clone().transpose(0, 1)
    assert out.shape == t.shape and out.stride() == (D, D, 1)
    return out


def test_one_token_heads_first():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([70], 2, 16)
    q = bf16_normal_bits(3, (1, 8, D))
    o = heads_first(torch.zeros(1, 8, D, dtype=torch.bfloat16, device="cuda"))
    got = rkv.attn_decode_paged(heads_first(to_dev(q)), st.cache, st.lens_dev, o=o)
    assert got is o
    check_decode(st, q, o, SCALE)
    kb, vb = bf16_normal_bits(4, (1, 2, D)), bf16_normal_bits(5, (1, 2, D))
    rkv.kvcache_paged_insert(st.cache, heads_first(to_dev(kb)), to_dev(vb), st.lens_dev)
    st.k[0][69], st.v[0][69] = kb[0], vb[0]
    check_decode(st, q, rkv.attn_decode_paged(to_dev(q), st.cache, st.lens_dev), SCALE)


def test_window_of_one_query_heads_first():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    q, k, v = (to_dev(bf16_normal_bits(10 + i, (n, h, D))) for i, (n, h) in enumerate(((1, 4), (300, 2), (300, 2))))
    rope, outs = rkv.make_rope(1, 1), []
    for view in (lambda t: t, heads_first):
        o = view(torch.zeros_like(q))
        s = rkv.AttnSeq(view(q), k, v, o, rope_q=False, rope_k=False, block_frames=1, q_frame_offset=299)
        rkv.rkv_attn_status(rkv.attn_fwd_window([s], [(100, 2)], rope))
        outs.append(o)
    assert torch.equal(*outs) and float(outs[0].abs().max()) > 0


def test_one_head_and_pages_of_one_token():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([40], 1, 1)
    q = bf16_normal_bits(3, (1, 2, D))
    want = rkv.attn_decode_paged(to_dev(q), st.cache, st.lens_dev)
    k, v = (t.reshape(-1, D) for t in (st.cache.k, st.cache.v))
    # [n_pages, 1, 1, D] as other views of the same rows
    k1, v1 = k[None, :, None].transpose(0, 1), v[None, None].permute(2, 0, 1, 3)
    assert k1.shape == st.cache.k.shape and k1.stride() != st.cache.k.stride()
    cache = rkv.PagedKVCache(k1, v1, st.cache.page_table)
    assert torch.equal(rkv.attn_decode_paged(to_dev(q), cache, st.lens_dev), want)
    check_decode(st, q, want, SCALE)


def test_one_page_a_sequence():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([9, 16, 3], 2, 16)
    table = st.cache.page_table.reshape(1, 3).clone().t()
    assert table.shape == (3, 1) and table.stride() == (1, 3)
    cache = rkv.PagedKVCache(st.cache.k, st.cache.v, table)
    q = bf16_normal_bits(3, (3, 2, D))
    check_decode(st, q, rkv.attn_decode_paged(to_dev(q), cache, st.lens_dev), SCALE)


def test_window_refuses_a_workspace_elsewhere():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    q, k, v = (to_dev(bf16_normal_bits(10 + i, (70, 2, D))) for i in range(3))
    s = rkv.AttnSeq(q, k, v, torch.empty_like(q), rope_q=False, rope_k=False, block_frames=1)
    big = 2 * rkv.attn_fwd_varlen_workspace_size()
    # (strided or on the host: refused before anything is launched)
    for ws in (torch.empty(big, dtype=torch.uint8), torch.empty(big, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            rkv.attn_fwd_window([s], [(3, 0)], rkv.make_rope(1, 1), workspace=ws)
