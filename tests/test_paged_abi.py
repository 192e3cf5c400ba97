"""The paged cache's calls without a GPU: struct layout and refusals on the host."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def rkv(lib_path):
    from rolling_kv_cache_rope_b200 import rkv as m
    return m


def cache(rkv, **kw):
    d = dict(k=0x100000000, v=0x200000000, page_stride=16 * 2 * 128, n_pages=40, page_tokens=16, H=2, D=128,
             page_table=0x300000000, table_stride=8, n_seqs=4, max_pages=8, status=0x310000000)
    d.update(kw)
    return rkv.rkv_paged_cache(**d)


BAD_CACHES = [
    (dict(k=0), "NULL"), (dict(v=0), "NULL"), (dict(page_table=0), "NULL"), (dict(D=64), "128"),
    (dict(n_pages=0), ">= 1"), (dict(page_tokens=0), ">= 1"), (dict(H=0), ">= 1"), (dict(n_seqs=0), ">= 1"),
    (dict(max_pages=0), ">= 1"), (dict(table_stride=7), "table_stride"), (dict(k=0x100000008), "aligned"),
    (dict(page_table=0x300000002), "aligned"), (dict(status=0x310000001), "aligned"),
    (dict(page_stride=16 * 2 * 128 - 128), "page_stride"), (dict(page_stride=16 * 2 * 128 + 8), "multiple"),
    (dict(v=0x100000000 + 4096), "overlap"),
]


def fake(x):
    return ctypes.c_void_p(x)


def insert(rkv, c, **kw):
    a = dict(k=0x400000000, v=0x410000000, stride=256, n=1, lens=0x500000000, nxt=0, pos=0, weight=0)
    a.update(kw)
    return rkv.lib().kvcache_paged_insert(ctypes.byref(c), fake(a["k"]), fake(a["v"]), a["stride"], a["n"],
                                          fake(a["lens"]), fake(a["nxt"]), fake(a["pos"]), fake(a["weight"]), None)


def decode(rkv, c, **kw):
    a = dict(q=0x400000000, o=0x410000000, qs=512, os=512, Hq=4, Lq=1, lens=0x500000000, scale=0.1, window=0, sinks=0,
             win=0, wout=0, ws=0x600000000, wsb=1 << 30)
    a.update(kw)
    return rkv.lib().attn_decode_paged(ctypes.byref(c), fake(a["q"]), fake(a["o"]), a["qs"], a["os"], a["Hq"], a["Lq"],
                                       fake(a["lens"]), a["scale"], a["window"], a["sinks"], fake(a["win"]),
                                       fake(a["wout"]), fake(a["ws"]), a["wsb"], None)


def evict(rkv, c, **kw):
    a = dict(lens=0x500000000, weight=0x510000000, pos=0x520000000, nxt=0x530000000, budget=10, sinks=1, recent=2,
             lens_out=0x500000000, wout=0x510000000, pout=0x520000000, ws=0x600000000, wsb=1 << 30)
    a.update(kw)
    return rkv.lib().kvcache_paged_evict(ctypes.byref(c), fake(a["lens"]), fake(a["weight"]), fake(a["pos"]),
                                         fake(a["nxt"]), a["budget"], a["sinks"], a["recent"], fake(a["lens_out"]),
                                         fake(a["wout"]), fake(a["pout"]), fake(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("change,frag", BAD_CACHES)
@pytest.mark.parametrize("call", [insert, decode, evict])
def test_bad_caches(rkv, call, change, frag):
    assert call(rkv, cache(rkv, **change)) == rkv.RKV_ERR_INVALID_ARG
    assert frag in rkv.rkv_last_error_string()


@pytest.mark.parametrize("call", [insert, decode, evict])
@pytest.mark.parametrize("change,frag", [
    (dict(n_pages=1 << 30, page_stride=16 * 2 * 128), "2^32"),
    (dict(max_pages=1 << 27, table_stride=1 << 27), "2^30"),
    (dict(page_tokens=1 << 30, H=2, page_stride=(1 << 31) * 128), "2^31"),
])
def test_caches_past_32_bits(rkv, call, change, frag):
    assert call(rkv, cache(rkv, **change)) == rkv.RKV_ERR_UNSUPPORTED
    assert frag in rkv.rkv_last_error_string()


def test_interleaved_pools_are_no_overlap(rkv):
    # k and v as the halves of one [n_pages][2][...] tensor
    half = 16 * 2 * 128
    c = cache(rkv, page_stride=2 * half, v=0x100000000 + 2 * half)
    assert insert(rkv, c, n=0) == rkv.RKV_OK
    # a source in the gap between two pages' halves is none either (the call gets as far as its
    # overlapping scores), one on a page is
    wide = cache(rkv, page_stride=4 * half, v=0x100000000 + 2 * half)
    scores = dict(nxt=0x700000000, pos=0x710000000, weight=0x710000004)
    assert insert(rkv, wide, k=0x100000000 + 4 * half, **scores) == rkv.RKV_ERR_INVALID_ARG
    assert "scores" in rkv.rkv_last_error_string()
    assert insert(rkv, wide, k=0x100000000 + 8 * half, **scores) == rkv.RKV_ERR_INVALID_ARG
    assert "new tokens" in rkv.rkv_last_error_string()


@pytest.mark.parametrize("change,frag", [
    (dict(n=-1), "n_new"), (dict(n=129), "n_new"), (dict(k=0), "NULL"), (dict(v=0), "NULL"), (dict(lens=0), "NULL"),
    (dict(pos=0x700000000), "together"), (dict(nxt=0x700000000), "together"), (dict(k=0x400000004), "aligned"),
    (dict(stride=128), "stride"), (dict(stride=260), "aligned"), (dict(stride=1 << 41), "stride"),
    (dict(k=0x100000000), "overlap"), (dict(v=0x200000000 + 64), "overlap"),
    (dict(weight=0x100000000), "overlap"), (dict(nxt=0x700000000, pos=0x200000000), "overlap"),
    (dict(nxt=0x700000000, pos=0x710000000, weight=0x710000004), "overlap"), (dict(lens=0x500000002), "4-byte"),
    (dict(nxt=0x700000000, pos=0x710000001), "4-byte"), (dict(weight=0x500000000), "overlap"),
    (dict(nxt=0x700000000, pos=0x700000000), "overlap"), (dict(weight=0x410000000), "overlap"),
])
def test_insert_rejects(rkv, change, frag):
    assert insert(rkv, cache(rkv), **change) == rkv.RKV_ERR_INVALID_ARG
    assert frag in rkv.rkv_last_error_string()


def test_insert_of_nothing_is_a_host_noop(rkv):
    assert insert(rkv, cache(rkv), n=0, k=0, v=0, lens=0) == rkv.RKV_OK


@pytest.mark.parametrize("change,frag", [
    (dict(Hq=3), "multiple"), (dict(Hq=0), "multiple"), (dict(Lq=0), "Lq"), (dict(Lq=65), "Lq"), (dict(q=0), "NULL"),
    (dict(o=0), "NULL"), (dict(lens=0), "NULL"), (dict(q=0x400000008), "aligned"), (dict(qs=256), "stride"),
    (dict(os=516), "aligned"), (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(window=-1), "window"), (dict(sinks=-1), "sinks"),
    (dict(win=0x700000000), "weight_out"), (dict(o=0x400000000), "overlap"), (dict(o=0x100000000), "overlap"),
    (dict(win=0x700000000, wout=0x700000010), "part"), (dict(wout=0x410000000), "overlap"),
    (dict(wout=0x200000000), "overlap"), (dict(lens=0x500000001), "4-byte"), (dict(wout=0x700000002), "4-byte"),
    (dict(lens=0x410000000), "overlap"), (dict(wout=0x500000000), "overlap"), (dict(ws=0), "workspace"), (dict(ws=0x600000008), "workspace"),
    (dict(wsb=16), "workspace"),
])
def test_decode_rejects(rkv, change, frag):
    assert decode(rkv, cache(rkv), **change) == rkv.RKV_ERR_INVALID_ARG
    assert frag in rkv.rkv_last_error_string()


def test_decode_too_many_rows(rkv):
    c = cache(rkv, H=1, page_stride=16 * 128)
    assert decode(rkv, c, Hq=128, Lq=64, qs=128 * 128, os=128 * 128) == rkv.RKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,frag", [
    (dict(lens=0), "NULL"), (dict(weight=0), "NULL"), (dict(pos=0), "NULL"), (dict(nxt=0), "NULL"),
    (dict(lens_out=0), "NULL"), (dict(wout=0), "NULL"), (dict(pout=0), "NULL"), (dict(budget=0), "budget"),
    (dict(sinks=-1), "sinks"), (dict(recent=-1), "recent"), (dict(wout=0x710000000), "both or neither"),
    (dict(wout=0x510000010, pout=0x720000000), "overlap"), (dict(wout=0x710000000, pout=0x710000010), "overlap"),
    (dict(wout=0x100000000, pout=0x720000000), "pool"), (dict(lens_out=0x500000004), "seq_lens_out"),
    (dict(lens_out=0x530000000), "seq_lens_out"), (dict(lens_out=0x100000000), "seq_lens_out"),
    (dict(pos=0x520000002, pout=0x520000002), "4-byte"), (dict(wout=0x530000000, pout=0x720000000), "overlap"), (dict(lens_out=0x510000040), "seq_lens_out"), (dict(ws=0), "workspace"), (dict(wsb=15), "workspace"),
])
def test_evict_rejects(rkv, change, frag):
    assert evict(rkv, cache(rkv), **change) == rkv.RKV_ERR_INVALID_ARG
    assert frag in rkv.rkv_last_error_string()


def test_workspace_sizes(rkv):
    lib = rkv.lib()
    c = cache(rkv)
    plain = lib.attn_decode_paged_workspace_size(ctypes.byref(c), 4, 1, 0)
    assert 0 < plain < lib.attn_decode_paged_workspace_size(ctypes.byref(c), 4, 1, 1)
    assert plain % 16 == 0
    assert lib.attn_decode_paged_workspace_size(ctypes.byref(c), 3, 1, 0) == 0
    assert lib.attn_decode_paged_workspace_size(None, 4, 1, 0) == 0
    assert lib.kvcache_paged_evict_workspace_size(ctypes.byref(c), 10) >= 4 * 2 * (1 + 2 * 10) * 4
    assert lib.kvcache_paged_evict_workspace_size(ctypes.byref(c), 0) == 0
    assert lib.rkv_paged_status(ctypes.byref(cache(rkv, status=0)), None) == rkv.RKV_ERR_INVALID_ARG


def test_python_cache_refuses_host_tensors(rkv):
    import torch
    k = torch.zeros(4, 8, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rkv.PagedKVCache(k, k.clone(), torch.zeros(1, 2, dtype=torch.int32))


@pytest.mark.parametrize("call", [insert, decode, evict])
def test_counts_past_64_bits(rkv, call):
    """2^30 key heads times 2^30 sequences: products of the counts would wrap around."""
    c = cache(rkv, H=1 << 30, n_seqs=1 << 30, page_tokens=1, n_pages=1, page_stride=128 << 30, max_pages=1,
              table_stride=1, k=1 << 52, v=1 << 53)
    assert call(rkv, c) == rkv.RKV_ERR_UNSUPPORTED
    assert "2^28" in rkv.rkv_last_error_string()
