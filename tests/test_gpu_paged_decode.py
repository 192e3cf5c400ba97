"""attn_decode_paged on the GPU against the float64 oracle.  Every row of the
pool that no query may see holds NaN, so a read outside the mask shows."""

import math

import numpy as np
import pytest
import torch

from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import need_gpu, to_bits, to_dev
from tests._paged import D, NAN, Streams, check_decode

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


def queries(st, Lq, G, seed=7):
    return bf16_normal_bits(seed, (st.n * Lq, st.H * G, D))


def run(st, q_bits, **kw):
    from rolling_kv_cache_rope_b200 import rkv
    o = torch.full(q_bits.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((max(16, rkv.attn_decode_paged_workspace_size(st.cache, q_bits.shape[1], q_bits.shape[0] // st.n,
                                                                  kw.get("weight_out") is not None)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    rkv.attn_decode_paged(to_dev(q_bits), st.cache, st.lens_dev, o=o, workspace=ws, **kw)
    rkv.rkv_paged_status(st.cache)
    return o


CASES = [
    # lens, H, G, P, Lq
    ([1], 1, 1, 1, 1),
    ([7], 2, 1, 4, 1),
    ([129], 3, 1, 16, 1),
    ([0], 2, 2, 16, 1),
    ([0, 1, 2, 0, 300, 17], 2, 4, 16, 1),
    ([128, 127, 16, 15], 1, 16, 8, 1),
    ([500, 3, 1951], 12, 1, 390, 1),
    ([1951], 12, 1, 390, 1),
    ([40, 5000], 1, 1, 1, 1),          # one key head, pages of one token, an item over many blocks
    ([4097], 2, 3, 24, 5),             # 15 rows
    ([900, 2], 2, 8, 100, 4),          # 32 rows
    ([300, 64, 9], 2, 8, 64, 8),       # 64 rows: two row blocks
    ([77, 310], 1, 7, 13, 7),          # 49 rows, the last row block half empty
    ([5, 3, 0], 1, 1, 16, 6),          # more queries than tokens
    ([700], 1, 33, 16, 1),             # 33 rows
    ([600], 4, 1, 1560, 1),            # one page, ending far past the length
    ([40001], 1, 1, 64, 1),            # an item over every block of the launch
    ([40001], 1, 2, 1560, 2),
]


@pytest.mark.parametrize("lens,H,G,P,Lq", CASES)
def test_decode(lens, H, G, P, Lq):
    need_gpu()
    st = Streams(lens, H, P)
    q = queries(st, Lq, G)
    check_decode(st, q, run(st, q), SCALE)


@pytest.mark.parametrize("lens,H,G,P,Lq", CASES)
def test_decode_weights(lens, H, G, P, Lq):
    need_gpu()
    st = Streams(lens, H, P, seed=3)
    q = queries(st, Lq, G)
    before = torch.rand(st.n, H, st.cap, device="cuda")
    after = torch.full_like(before, -5.0)
    o = run(st, q, weight_in=before, weight_out=after)
    check_decode(st, q, o, SCALE, w_before=before.cpu().numpy(), w_after=after.cpu().numpy())
    for s, L in enumerate(lens):
        assert torch.all(after[s, :, L:] == -5.0)       # left as it was
    inplace = before.clone()
    o2 = run(st, q, weight_in=inplace, weight_out=inplace)
    assert torch.equal(o, o2)
    for s, L in enumerate(lens):
        assert torch.equal(inplace[s, :, :L], after[s, :, :L]) and torch.equal(inplace[s, :, L:], before[s, :, L:])
    alone = torch.zeros_like(before)
    run(st, q, weight_out=alone)
    check_decode(st, q, o, SCALE, w_after=alone.cpu().numpy())
    # the outputs without the weights are the same bits
    assert torch.equal(run(st, q), o)


@pytest.mark.parametrize("lens,H,G,P,Lq,window,sinks", [
    ([700], 2, 2, 16, 1, 100, 4),
    ([700, 50, 99, 100, 101, 0], 1, 1, 16, 1, 100, 4),
    ([3000, 20], 2, 1, 24, 4, 513, 70),
    ([300], 1, 4, 7, 6, 1, 0),
    ([300], 1, 4, 7, 6, 1, 3),
    ([2000], 1, 1, 64, 3, 64, 1999),
    ([64, 1000], 2, 8, 32, 5, 130, 129),   # 40 rows
    ([900], 1, 2, 16, 8, 5, 0),            # windows that end between the queries
])
def test_decode_window(lens, H, G, P, Lq, window, sinks):
    need_gpu()
    st = Streams(lens, H, P, seed=5)
    # tokens no query sees hold NaN and infinities
    for s, L in enumerate(lens):
        first = max(0, max(0, L - Lq) - window + 1)
        hidden = slice(min(sinks, first), first)
        pg, tk = (torch.from_numpy(np.ascontiguousarray(x[hidden])).long().cuda() for x in st.rows(s))
        st.cache.k[pg, tk] = float("nan")
        st.cache.v[pg, tk] = float("inf")
    q = queries(st, Lq, G)
    before = torch.rand(st.n, H, st.cap, device="cuda")
    after = torch.empty_like(before)
    o = run(st, q, window=window, sinks=sinks, weight_in=before, weight_out=after)
    check_decode(st, q, o, SCALE, window, sinks, before.cpu().numpy(), after.cpu().numpy())
    assert torch.equal(run(st, q, window=window, sinks=sinks), o)


def test_many_short_streams():
    need_gpu()
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 40, 700)]
    st = Streams(lens, 2, 16, seed=9)
    q = queries(st, 1, 2)
    after = torch.zeros(st.n, 2, st.cap, device="cuda")
    o = run(st, q, weight_out=after)
    check_decode(st, q, o, SCALE, w_after=after.cpu().numpy())


def test_growing_maximum_and_scale():
    # scores that grow along the stream by far more than 2^8 move the running maximum again and again
    need_gpu()
    st = Streams([2100], 1, 16, seed=2)
    q = queries(st, 1, 1)
    o = run(st, q, softmax_scale=1.5)
    check_decode(st, q, o, 1.5)


def test_strides_interleaved_pool_and_guards():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([33, 130], 2, 16, interleaved=True, cols=12, table_pad=5)
    q_bits = queries(st, 2, 3)
    wide = torch.full((4, 9, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = to_dev(q_bits)
    out = torch.full((6, 8, D), -3.0, dtype=torch.bfloat16, device="cuda")
    o = out[1:5, 1:7]
    rkv.attn_decode_paged(wide[:, 2:8], st.cache, st.lens_dev, o=o)
    check_decode(st, q_bits, o.contiguous(), SCALE)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:5, 1:7] = False
    assert torch.all(out[keep] == -3.0)


def test_shared_pages_and_repeat():
    # two streams over the same pages, and the same bits every time
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([1000], 2, 16)
    table = st.cache.page_table.repeat(2, 1)
    two = rkv.PagedKVCache(st.cache.k, st.cache.v, table)
    lens = torch.tensor([1000, 700], dtype=torch.int32, device="cuda")
    q_bits = bf16_normal_bits(4, (2, 4, D))
    o = rkv.attn_decode_paged(to_dev(q_bits), two, lens)
    st.lens, st.k, st.v = [1000, 700], [st.k[0], st.k[0][:700]], [st.v[0], st.v[0][:700]]
    check_decode(st, q_bits, o, SCALE)
    for _ in range(5):
        assert torch.equal(rkv.attn_decode_paged(to_dev(q_bits), two, lens), o)


def test_lengths_and_pages_out_of_range():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([64, 50, 40], 2, 16, cols=4)
    q = queries(st, 1, 2)
    o = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(3, 2, 64, device="cuda")
    # a negative length is an empty stream, one past the capacity the capacity
    bad = torch.tensor([1 << 30, 50, -9], dtype=torch.int32, device="cuda")
    rkv.attn_decode_paged(to_dev(q), st.cache, bad, o=o, weight_out=w)
    with pytest.raises(rkv.RkvError, match="length") as e:
        rkv.rkv_paged_status(st.cache)
    assert e.value.status == rkv.RKV_ERR_DEVICE_CHECK
    rkv.rkv_paged_status(st.cache)       # cleared
    st.lens, st.k[2], st.v[2] = [64, 50, 0], st.k[2][:0], st.v[2][:0]
    check_decode(st, q, o, SCALE, w_after=w.cpu().numpy())
    # tokens on a page outside the pool are not visible
    st = Streams([64, 50], 1, 16, cols=4)
    st.cache.page_table[0, 1] = 1 << 20
    st.cache.page_table[1, 0] = -1
    q = queries(st, 1, 2)
    w = torch.zeros(2, 1, 64, device="cuda")
    o = rkv.attn_decode_paged(to_dev(q), st.cache, st.lens_dev, weight_out=w)
    with pytest.raises(rkv.RkvError, match="page"):
        rkv.rkv_paged_status(st.cache)
    assert torch.all(w[0, 0, 16:32] == 0) and torch.all(w[1, 0, :16] == 0)
    assert torch.allclose(w.sum(-1).cpu(), torch.full((2, 1), 2.0), atol=1e-5)
    keep = [np.r_[0:16, 32:64], np.r_[16:50]]
    st.k, st.v = [st.k[s][keep[s]] for s in (0, 1)], [st.v[s][keep[s]] for s in (0, 1)]
    check_decode(st, q, o, SCALE)


def test_other_stream_and_captured_launch():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([300, 260], 2, 16, cols=40)
    q_bits = queries(st, 1, 2)
    q = to_dev(q_bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = rkv.attn_decode_paged(q, st.cache, st.lens_dev, stream=side)
    side.synchronize()
    check_decode(st, q_bits, o, SCALE)
    # two captured launches, each with its own workspace, replayed while the streams' lengths change
    graphs = []
    for _ in range(2):
        out, w = torch.zeros_like(o), torch.zeros(2, 2, st.cap, device="cuda")
        ws = torch.empty(rkv.attn_decode_paged_workspace_size(st.cache, 4, 1, True), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rkv.attn_decode_paged(q, st.cache, st.lens_dev, o=out, weight_out=w, workspace=ws)
        graphs.append((g, out, w))
    for lens in ([300, 260], [150, 1], [0, 259]):
        st.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        for g, _, w in graphs:
            w.zero_()
            g.replay()
        torch.cuda.synchronize()
        view = Streams.__new__(Streams)
        view.__dict__.update(st.__dict__, lens=lens, k=[st.k[s][:lens[s]] for s in (0, 1)],
                             v=[st.v[s][:lens[s]] for s in (0, 1)])
        for _, out, w in graphs:
            check_decode(view, q_bits, out, SCALE, w_after=w.cpu().numpy())


def test_offsets_past_32_bits():
    # a pool of more than 2^32 bytes, the stream's pages at its end
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    H, P, n_pages = 8, 64, 36000     # 36000 * 64 * 8 * 256 B = 4.7 GB each
    k = torch.empty(n_pages, P, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    st = Streams([777], H, P, seed=6)
    used = -(-777 // P)
    table = torch.arange(n_pages - used, n_pages, dtype=torch.int32, device="cuda").flip(0).view(1, used)
    src = st.cache.page_table[0].long()
    k[table[0].long()] = st.cache.k[src]
    v[table[0].long()] = st.cache.v[src]
    q = queries(st, 1, 1)
    o = rkv.attn_decode_paged(to_dev(q), rkv.PagedKVCache(k, v, table), st.lens_dev)
    check_decode(st, q, o, SCALE)


def test_over_a_ring():
    # a ring's buffers are a pool whose pages are frames: decode over its valid frames, oldest first
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    H, F, W = 2, 24, 5
    ring = rkv.KVRing(W, F, H)
    ring.k.fill_(float("nan"))
    ring.v.fill_(float("nan"))
    st = Streams([0], H, F)
    kb, vb = bf16_normal_bits(1, (7 * F, H, D)), bf16_normal_bits(2, (7 * F, H, D))
    for f0, n in ((0, 4), (4, 3)):
        rkv.kvcache_ring_update(ring, to_dev(kb[f0 * F:(f0 + n) * F]), to_dev(vb[f0 * F:(f0 + n) * F]), n)
    table = torch.tensor([[ring.slot(j) for j in range(ring.count)]], dtype=torch.int32, device="cuda")
    cache = rkv.PagedKVCache(ring.k, ring.v, table)
    L = ring.valid_rows()
    q = bf16_normal_bits(3, (1, H, D))
    o = rkv.attn_decode_paged(to_dev(q), cache, torch.tensor([L], dtype=torch.int32, device="cuda"), window=50, sinks=3)
    st.lens, st.k, st.v = [L], [kb[2 * F:]], [vb[2 * F:]]
    check_decode(st, q, o, SCALE, 50, 3)


def test_python_refusals():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([30], 2, 16)
    q = to_dev(queries(st, 1, 1))
    c = st.cache
    with pytest.raises(ValueError, match="seq_lens"):
        rkv.attn_decode_paged(q, c, st.lens_dev.long())
    with pytest.raises(ValueError, match="seq_lens"):
        rkv.attn_decode_paged(q, c, st.lens_dev.cpu())
    with pytest.raises(ValueError, match="weight_out"):
        rkv.attn_decode_paged(q, c, st.lens_dev, weight_out=torch.zeros(1, 2, 31, device="cuda"))
    with pytest.raises(ValueError, match="o must be"):
        rkv.attn_decode_paged(q, c, st.lens_dev, o=torch.empty(2, 2, D, dtype=q.dtype, device="cuda"))
    with pytest.raises(rkv.RkvError, match="workspace"):
        rkv.attn_decode_paged(q, c, st.lens_dev, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="page_table"):
        rkv.PagedKVCache(c.k, c.v, c.page_table.long())
    with pytest.raises(ValueError, match="contiguous"):
        rkv.PagedKVCache(c.k.transpose(1, 2), c.v.transpose(1, 2), c.page_table)
    assert to_bits(q).shape == (1, 2, D) and NAN


def test_largest_rows():
    # RKV_DECODE_MAX_LQ queries of two heads to a key head
    need_gpu()
    st = Streams([200, 63], 1, 16)
    q = queries(st, 64, 2)
    after = torch.zeros(2, 1, st.cap, device="cuda")
    o = run(st, q, window=40, sinks=2, weight_out=after)
    check_decode(st, q, o, SCALE, 40, 2, None, after.cpu().numpy())


def test_window_and_sinks_at_their_largest():
    need_gpu()
    st = Streams([5, 900], 2, 16)
    q = queries(st, 8, 2)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        o = run(st, q, window=window, sinks=sinks)
        check_decode(st, q, o, SCALE, window, sinks)


def test_two_calls_at_once():
    # two streams over one cache, each call with its own workspace, again and again
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([3000, 10, 700], 2, 16)
    qs = [queries(st, 1, 4, seed=s) for s in (1, 2)]
    devs = [to_dev(q) for q in qs]
    want = [run(st, q) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(rkv.attn_decode_paged(devs[i], st.cache, st.lens_dev, stream=s))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_calls_in_a_row_without_waiting():
    # each call reads what the one before wrote (lengths, weights, queries), with nothing in between
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([600, 90], 2, 16)
    q_bits = queries(st, 1, 2)
    q = to_dev(q_bits)
    w, lens = torch.zeros(2, 2, st.cap, device="cuda"), st.lens_dev.clone()
    ws = torch.empty(rkv.attn_decode_paged_workspace_size(st.cache, 4, 1, True), dtype=torch.uint8, device="cuda")
    one = torch.zeros_like(w)
    rkv.attn_decode_paged(q, st.cache, lens, weight_out=one, workspace=ws)
    o = q
    for _ in range(20):
        o = rkv.attn_decode_paged(q, st.cache, lens, weight_in=w, weight_out=w, workspace=ws)
    want = torch.zeros_like(w)
    for _ in range(20):
        want = want + one
    assert torch.equal(w, want)
    check_decode(st, q_bits, o, SCALE)
