"""kvcache_paged_insert and kvcache_paged_evict on the GPU: bit-exact against
the oracle, everything outside the written places unchanged; and the calls of a
bounded stream's step together."""

import math

import numpy as np
import pytest
import torch

from oracle import bf16_bits_to_f64, evict_moves
from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import need_gpu, to_dev
from tests._paged import D, Streams, check_decode

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("lens,H,P,new,scores,interleaved", [
    ([1], 1, 1, 1, True, False),
    ([40, 1, 0, 17], 3, 16, 1, True, False),
    ([5, 3, 0, 200], 2, 7, 4, True, True),       # a stream shorter than the insert, an empty one
    ([390, 391, 1000], 12, 390, 390, True, False),
    ([64, 64], 8, 64, 64, False, True),
    ([33], 2, 1560, 20, True, False),
])
def test_insert(lens, H, P, new, scores, interleaved):
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams(lens, H, P, interleaved=interleaved)
    n = st.n
    kb, vb = bf16_normal_bits(50, (n * new, H, D)), bf16_normal_bits(51, (n * new, H, D))
    wide = torch.zeros(n * new, H + 2, D, dtype=torch.bfloat16, device="cuda")
    wide2 = torch.zeros_like(wide)
    wide[:, 1:-1], wide2[:, 1:-1] = to_dev(kb), to_dev(vb)
    before = [bits(st.cache.k).clone(), bits(st.cache.v).clone()]
    nxt = st.lens_dev + 500
    pos = torch.full((n, H, st.cap), -1, dtype=torch.int32, device="cuda")
    weight = torch.full((n, H, st.cap), 2.5, device="cuda")
    kw = dict(next_pos=nxt, pos=pos, weight=weight) if scores else {}
    rkv.kvcache_paged_insert(st.cache, wide[:, 1:-1], wide2[:, 1:-1], st.lens_dev, **kw)
    rkv.rkv_paged_status(st.cache)
    want_pos, want_w = np.full((n, H, st.cap), -1), np.full((n, H, st.cap), 2.5)
    for s, L in enumerate(lens):
        pg, tk = st.rows(s)
        for i in range(new):
            j = L - new + i
            if j < 0:
                continue
            for t, src in zip(before, (kb, vb)):
                t[pg[j], tk[j]] = torch.from_numpy(src[s * new + i].view(np.int16)).cuda()
            want_pos[s, :, j], want_w[s, :, j] = L + 500 - new + i, 0.0
    assert torch.equal(bits(st.cache.k), before[0]) and torch.equal(bits(st.cache.v), before[1])
    if scores:
        assert np.array_equal(pos.cpu().numpy(), want_pos) and np.array_equal(weight.cpu().numpy(), want_w)


def test_insert_out_of_range():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([10, 30, 5], 2, 16, cols=2)
    kb = bf16_normal_bits(1, (3, 2, D))
    before = bits(st.cache.k).clone()
    st.cache.page_table[0, 0] = st.cache.k.shape[0]     # one past the pool
    rkv.kvcache_paged_insert(st.cache, to_dev(kb), to_dev(kb), torch.tensor([10, -1, 0], dtype=torch.int32, device="cuda"))
    with pytest.raises(rkv.RkvError, match="RKV_ERR_DEVICE_CHECK"):
        rkv.rkv_paged_status(st.cache)
    assert torch.equal(bits(st.cache.k), before)
    # a length past the capacity: the last token of the capacity
    st = Streams([32], 1, 16, cols=2)
    rkv.kvcache_paged_insert(st.cache, to_dev(kb[:1, :1]), to_dev(kb[:1, :1]),
                             torch.tensor([1000], dtype=torch.int32, device="cuda"))
    with pytest.raises(rkv.RkvError, match="length"):
        rkv.rkv_paged_status(st.cache)
    assert np.array_equal(st.gathered(0)[0][31], kb[0, :1])


def evict_case(lens, H, P, budget, sinks, recent, weight, pos, nxt, in_place, cols=None, table_of=None):
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams(lens, H, P, seed=11, cols=cols)
    n, cap = st.n, st.cap
    w0 = np.full((n, H, cap), 9.0, dtype=np.float32)
    p0 = np.full((n, H, cap), -9, dtype=np.int32)
    for s, L in enumerate(lens):
        w0[s, :, :L], p0[s, :, :L] = weight(s, L), pos(s, L)
    w, p = torch.from_numpy(w0).cuda(), torch.from_numpy(p0).cuda()
    nx = torch.tensor([nxt(s, L) for s, L in enumerate(lens)], dtype=torch.int32, device="cuda")
    k0, v0 = bits(st.cache.k).clone(), bits(st.cache.v).clone()
    lens_in = st.lens_dev.clone()
    if in_place:
        rkv.kvcache_paged_evict(st.cache, lens_in, w, p, nx, budget, sinks, recent)
        wo, po, lo = w, p, lens_in
        want_w, want_p = w0.copy(), p0.copy()
    else:
        wo, po, lo = torch.full_like(w, 5.0), torch.full_like(p, 5), torch.full_like(lens_in, -1)
        ws = torch.full((max(16, rkv.kvcache_paged_evict_workspace_size(st.cache, budget)),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        rkv.kvcache_paged_evict(st.cache, lens_in, w, p, nx, budget, sinks, recent, seq_lens_out=lo, weight_out=wo,
                                pos_out=po, workspace=ws)
        assert np.array_equal(w.cpu().numpy(), w0, equal_nan=True) and np.array_equal(p.cpu().numpy(), p0)
        assert torch.equal(lens_in, st.lens_dev)
        want_w, want_p = np.full_like(w0, 5.0), np.full_like(p0, 5)
        for s, L in enumerate(lens):
            m = min(L, budget)
            want_w[s, :, :m], want_p[s, :, :m] = w0[s, :, :m], p0[s, :, :m]
    rkv.rkv_paged_status(st.cache)
    moved = 0
    for s, L in enumerate(lens):
        pg, tk = st.rows(s)
        for h in range(H):
            for a, b in evict_moves(w0[s, h, :L], p0[s, h, :L], nxt(s, L), budget, sinks, recent):
                want_w[s, h, b], want_p[s, h, b] = w0[s, h, a], p0[s, h, a]
                k0[pg[b], tk[b], h] = k0[pg[a], tk[a], h]
                v0[pg[b], tk[b], h] = v0[pg[a], tk[a], h]
                moved += 1
    assert lo.tolist() == [min(L, budget) for L in lens]
    assert np.array_equal(po.cpu().numpy(), want_p)
    assert np.array_equal(wo.cpu().numpy().view(np.int32), want_w.view(np.int32))
    assert torch.equal(bits(st.cache.k), k0) and torch.equal(bits(st.cache.v), v0)
    return moved


def normal_weight(seed):
    return lambda s, L: np.random.default_rng(seed + s).exponential(size=(1, L)) * np.ones((1, 1))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,H,P,budget,sinks,recent", [
    ([1], 1, 1, 1, 0, 0),
    ([2], 1, 1, 1, 0, 0),
    ([2], 1, 1, 1, 0, 1),
    ([100, 0, 64, 65, 1], 3, 16, 64, 4, 16),
    ([513], 2, 24, 512, 4, 100),
    ([513], 2, 24, 512, 0, 0),
    ([700, 2000], 2, 100, 300, 1, 299),
    ([700, 2000], 2, 100, 300, 300, 0),
    ([700], 1, 390, 300, 200, 250),          # more protected than the budget: the first of them stay
    ([1024], 4, 32, 1023, 4, 64),
    ([4097], 2, 1560, 17, 2, 5),
    ([90, 88], 2, 7, 80, 2, 9),              # scores that do not start on 16-byte boundaries
    ([2050, 90], 1, 13, 2033, 2, 9),
])
def test_evict(lens, H, P, budget, sinks, recent, in_place):
    need_gpu()
    rng = np.random.default_rng(budget)
    order = [np.stack([rng.permutation(L) for _ in range(H)]) if L else np.zeros((H, 0)) for L in lens]
    weights = [rng.exponential(size=(H, L)).astype(np.float32) for L in lens]
    evict_case(lens, H, P, budget, sinks, recent, lambda s, L: weights[s], lambda s, L: order[s], lambda s, L: L, in_place)


@pytest.mark.parametrize("values", [
    [0.0], [0.0, 1.0], [0.0, -0.0, 1e-45], [float("inf"), 1.0, float("-inf"), -1.0, 0.0],
    [float("nan"), 0.0, float("inf")], [float("nan")], [1.0, 1.0000001, 0.9999999],
])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_ties_and_special_weights(values, in_place):
    need_gpu()
    rng = np.random.default_rng(len(values))
    L, H = 1500, 2
    w = rng.choice(np.array(values, dtype=np.float32), size=(H, L))
    evict_case([L], H, 16, 700, 3, 50, lambda s, n: w, lambda s, n: np.tile(np.arange(L), (H, 1)), lambda s, n: L, in_place)


def test_evict_long_streams():
    # more tokens than the keys of one head that fit shared memory, and positions at the ends of int32
    need_gpu()
    L = 60001
    rng = np.random.default_rng(8)
    w = np.round(rng.exponential(size=(1, L)), 2).astype(np.float32)
    p = np.arange(L)[None] + (2 ** 31 - 1 - L)
    assert evict_case([L], 1, 64, 20000, 0, 1000, lambda s, n: w, lambda s, n: p, lambda s, n: 2 ** 31 - 1, False) > 1000
    p = np.arange(L)[None] - 2 ** 31
    evict_case([L], 1, 64, 59999, 5, 2 ** 31 - 1, lambda s, n: w, lambda s, n: p, lambda s, n: -(2 ** 31), True)


@pytest.mark.parametrize("L,H,n,budget,sinks,recent,ties", [
    (9000, 1, 1, 4000, 7, 100, 0), (17001, 2, 1, 16999, 0, 0, 0), (17001, 2, 2, 5, 1, 1, 0), (33000, 3, 1, 20000, 500, 9000, 0),
    (9000, 1, 1, 4000, 7, 100, 3), (33000, 1, 2, 16384, 0, 2000, 2), (8192, 5, 3, 8000, 0, 0, 1),
])
def test_evict_few_long_heads(L, H, n, budget, sinks, recent, ties):
    # few heads of many tokens: each shared out over a cluster of blocks
    need_gpu()
    rng = np.random.default_rng(L + ties)
    w = rng.exponential(size=(n, H, L)).astype(np.float32)
    if ties:
        w = np.floor(w * ties)
    lens = [L - 3 * s for s in range(n)]
    order = [np.stack([rng.permutation(x) for _ in range(H)]) for x in lens]
    evict_case(lens, H, 64, budget, sinks, recent, lambda s, x: w[s, :, :x], lambda s, x: order[s], lambda s, x: x, bool(ties))


def test_evict_capacity_below_budget():
    need_gpu()
    assert evict_case([30, 5], 2, 16, 4000, 1, 5, lambda s, L: np.ones((2, L)), lambda s, L: np.tile(np.arange(L), (2, 1)),
                      lambda s, L: L, False) == 0


def test_evict_bad_pages_and_lengths():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([64, 20, 8], 1, 16, cols=4)
    k0 = bits(st.cache.k).clone()
    w = torch.arange(64, device="cuda", dtype=torch.float32).repeat(3, 1, 1)
    p = torch.arange(64, device="cuda", dtype=torch.int32).repeat(3, 1, 1)
    lens = torch.tensor([64, -5, 1 << 20], dtype=torch.int32, device="cuda")
    good = st.cache.page_table.clone()
    st.cache.page_table[0, 3] = -1           # the heaviest tokens of stream 0 lie on it
    st.cache.page_table[2] = st.cache.page_table[0]
    nxt = torch.full((3,), 64, dtype=torch.int32, device="cuda")
    rkv.kvcache_paged_evict(st.cache, lens, w, p, nxt, 16)
    with pytest.raises(rkv.RkvError, match="RKV_ERR_DEVICE_CHECK"):
        rkv.rkv_paged_status(st.cache)
    assert torch.equal(bits(st.cache.k), k0)     # nothing moved from or to the bad page, nothing else moves
    assert lens.tolist() == [16, 0, 16]
    assert good.shape == (3, 4)


def test_evict_captured():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams([200], 2, 16)
    w = torch.rand(1, 2, st.cap, device="cuda")
    p = torch.arange(st.cap, dtype=torch.int32, device="cuda").repeat(1, 2, 1).contiguous()
    nxt = torch.tensor([200], dtype=torch.int32, device="cuda")
    ws = torch.empty(rkv.kvcache_paged_evict_workspace_size(st.cache, 150), dtype=torch.uint8, device="cuda")
    lens = st.lens_dev.clone()
    w0, p0, k0 = w.clone(), p.clone(), st.cache.k.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rkv.kvcache_paged_evict(st.cache, lens, w, p, nxt, 150, 4, 20, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    first = (w.clone(), p.clone(), st.cache.k.clone())
    assert lens.tolist() == [150]
    w.copy_(w0), p.copy_(p0), st.cache.k.copy_(k0), lens.fill_(200)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, first[0]) and torch.equal(p, first[1])
    assert torch.equal(bits(st.cache.k), bits(first[2]))


def test_bounded_stream():
    """Insert, attend with weights, evict, step by step: every call against the
    oracle on the streams as the host keeps them."""
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    H, G, P, budget, sinks, recent, steps = 2, 2, 16, 40, 2, 8, 12
    start = [39, 17, 40]
    n = len(start)
    st = Streams(start, H, P, cols=3)          # capacity 48
    # the pages every stream will need, all listed from the start
    need = 3 * n
    pool = torch.full((need, P, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = pool.clone(), pool.clone()
    table = torch.randperm(need, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(n, 3).cuda()
    for s in range(n):
        for c in range(-(-start[s] // P)):
            k[table[s, c].long()] = st.cache.k[st.cache.page_table[s, c].long()]
            v[table[s, c].long()] = st.cache.v[st.cache.page_table[s, c].long()]
    cache = rkv.PagedKVCache(k, v, table)
    st.cache, st.table = cache, table.cpu().numpy()
    weight = torch.zeros(n, H, cache.capacity, device="cuda")
    pos = torch.arange(cache.capacity, dtype=torch.int32, device="cuda").repeat(n, H, 1).contiguous()
    lens, nxt = st.lens_dev.clone(), st.lens_dev.clone()
    # host side: per stream and head, rows in cache order
    hk = [st.k[s].copy() for s in range(n)]
    hv = [st.v[s].copy() for s in range(n)]
    for step in range(steps):
        new = 1 if step % 3 else 2
        kb, vb = bf16_normal_bits(100 + step, (n * new, H, D)), bf16_normal_bits(200 + step, (n * new, H, D))
        lens += new
        nxt += new
        rkv.kvcache_paged_insert(cache, to_dev(kb), to_dev(vb), lens, next_pos=nxt, pos=pos, weight=weight)
        hk = [np.concatenate([hk[s], kb[s * new:(s + 1) * new]]) for s in range(n)]
        hv = [np.concatenate([hv[s], vb[s * new:(s + 1) * new]]) for s in range(n)]
        st.lens, st.k, st.v = [len(x) for x in hk], hk, hv
        q = bf16_normal_bits(300 + step, (n * new, H * G, D))
        before = weight.cpu().numpy()
        o = rkv.attn_decode_paged(to_dev(q), cache, lens, weight_in=weight, weight_out=weight)
        check_decode(st, q, o, 1 / math.sqrt(D), w_before=before, w_after=weight.cpu().numpy())
        w, p, nx = weight.cpu().numpy(), pos.cpu().numpy(), nxt.tolist()
        rkv.kvcache_paged_evict(cache, lens, weight, pos, nxt, budget, sinks, recent)
        rkv.rkv_paged_status(cache)
        for s in range(n):
            L = st.lens[s]
            hk[s], hv[s] = hk[s].copy(), hv[s].copy()
            for h in range(H):
                for a, b in evict_moves(w[s, h, :L], p[s, h, :L], nx[s], budget, sinks, recent):
                    hk[s][b, h], hv[s][b, h] = hk[s][a, h], hv[s][a, h]
                    w[s, h, b], p[s, h, b] = w[s, h, a], p[s, h, a]
            m = min(L, budget)
            hk[s], hv[s] = hk[s][:m], hv[s][:m]
            assert np.array_equal(weight.cpu().numpy()[s, :, :m], w[s, :, :m])
            assert np.array_equal(pos.cpu().numpy()[s, :, :m], p[s, :, :m])
            # sinks and the newest tokens are all there
            for h in range(H):
                assert {0, 1} | set(range(max(0, nx[s] - recent), nx[s])) <= set(p[s, h, :m].tolist())
        st.lens = [len(x) for x in hk]
        assert lens.tolist() == st.lens
        for s in range(n):
            gk, gv = st.gathered(s)
            assert np.array_equal(gk, hk[s]) and np.array_equal(gv, hv[s])
    assert np.isfinite(bf16_bits_to_f64(hk[0])).all()
