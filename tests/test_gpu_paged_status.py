"""The status word of a cache that is used on another stream than the one it was
made on."""

import pytest
import torch

from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import need_gpu, to_dev
from tests._paged import D, Streams

pytestmark = pytest.mark.gpu


def test_finding_on_another_stream_is_kept():
    """The cache is made while its stream is busy; a call on a side stream then meets a bad length."""
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([30, 20], 2, 16)
    q = to_dev(bf16_normal_bits(3, (2, 2, D)))
    o, lens = torch.empty_like(q), torch.tensor([-4, 20], dtype=torch.int32, device="cuda")
    ws = torch.empty(rkv.attn_decode_paged_workspace_size(st.cache, 2), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    rkv.attn_decode_paged(q, st.cache, st.lens_dev, o=o, workspace=ws, stream=side)    # everything loaded
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(100_000_000)       # about 50 ms of the current stream
        cache = rkv.PagedKVCache(st.cache.k, st.cache.v, st.cache.page_table)
        rkv.attn_decode_paged(q, cache, lens, o=o, workspace=ws, stream=side)
        torch.cuda.synchronize()
        with pytest.raises(rkv.RkvError, match="length"):
            rkv.rkv_paged_status(cache, stream=side)
        rkv.rkv_paged_status(cache)


def test_fresh_cache_reports_nothing_on_another_stream():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([30], 2, 16)
    side = torch.cuda.Stream()
    for _ in range(20):                      # freed words of ones are what the next cache's word is made of
        junk = [torch.full((1,), 0x0101, dtype=torch.int32, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        torch.cuda._sleep(5_000_000)
        cache = rkv.PagedKVCache(st.cache.k, st.cache.v, st.cache.page_table)
        rkv.rkv_paged_status(cache, stream=side)
        torch.cuda.synchronize()


def test_cache_made_for_a_captured_call():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([30, 20], 2, 16)
    q = to_dev(bf16_normal_bits(3, (2, 2, D)))
    o, lens = torch.empty_like(q), torch.tensor([30, 20], dtype=torch.int32, device="cuda")
    ws = torch.empty(rkv.attn_decode_paged_workspace_size(st.cache, 2), dtype=torch.uint8, device="cuda")
    rkv.attn_decode_paged(q, st.cache, lens, o=o, workspace=ws)
    want = o.clone()
    cache = rkv.PagedKVCache(st.cache.k, st.cache.v, st.cache.page_table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):                # a stream of its own, the cache's first call
        rkv.attn_decode_paged(q, cache, lens, o=o, workspace=ws)
    o.zero_()
    g.replay()
    rkv.rkv_paged_status(cache)
    assert torch.equal(o, want)
    lens[0] = 1000
    g.replay()
    with pytest.raises(rkv.RkvError, match="length"):
        rkv.rkv_paged_status(cache)
