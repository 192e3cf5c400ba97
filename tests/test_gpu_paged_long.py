"""Evictions of streams with more keys than a block's shared memory holds, and
attention over an evicted cache."""

import math

import numpy as np
import pytest
import torch

from oracle import evict_moves
from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import need_gpu, to_dev
from tests._paged import D, Streams, check_decode

pytestmark = pytest.mark.gpu


def moves_of(w, p, nxt, budget, sinks, recent):
    """evict_moves by a stable sort: its moves (source, destination) as two arrays."""
    L = len(w)
    safe = (p < sinks) | (p.astype(np.int64) >= nxt - recent)
    order = np.argsort(np.where(safe, -np.inf, -w.astype(np.float64)), kind="stable")
    kept = np.zeros(L, dtype=bool)
    kept[order[:budget]] = True
    return budget + np.nonzero(kept[budget:])[0], np.nonzero(~kept[:budget])[0]


def evict_long(L, H, P, budget, sinks, recent, ties, in_place):
    from rolling_kv_cache_rope_b200 import rkv
    cols = -(-L // P)
    gen = torch.Generator(device="cuda").manual_seed(L + ties)
    k, v = (torch.randint(-32768, 32768, (cols, P, H, D), dtype=torch.int16, device="cuda", generator=gen) for _ in range(2))
    table = torch.randperm(cols, device="cuda", generator=gen).to(torch.int32).view(1, cols)
    cache = rkv.PagedKVCache(k.view(torch.bfloat16), v.view(torch.bfloat16), table)
    rng = np.random.default_rng(L)
    w0 = rng.exponential(size=(1, H, cols * P)).astype(np.float32)
    if ties:
        w0 = np.floor(w0 * ties)
    p0 = np.stack([rng.permutation(cols * P) for _ in range(H)])[None].astype(np.int32)
    w, p = torch.from_numpy(w0).cuda(), torch.from_numpy(p0).cuda()
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    nxt = torch.tensor([L], dtype=torch.int32, device="cuda")
    want = [k.clone(), v.clone()]
    kw = {} if in_place else dict(seq_lens_out=torch.zeros_like(lens), weight_out=torch.full_like(w, 5.0),
                                  pos_out=torch.full_like(p, 5))
    rkv.kvcache_paged_evict(cache, lens, w, p, nxt, budget, sinks, recent, **kw)
    rkv.rkv_paged_status(cache)
    got_w, got_p = (w, p) if in_place else (kw["weight_out"], kw["pos_out"])
    want_w, want_p = (w0.copy(), p0.copy()) if in_place else (np.full_like(w0, 5.0), np.full_like(p0, 5))
    want_w[:, :, :budget], want_p[:, :, :budget] = w0[:, :, :budget], p0[:, :, :budget]
    table_host = table[0].cpu().numpy()
    moved = 0
    for h in range(H):
        a, b = moves_of(w0[0, h, :L], p0[0, h, :L], L, budget, sinks, recent)
        if h == 0:
            assert list(zip(a, b)) == evict_moves(w0[0, h, :L], p0[0, h, :L], L, budget, sinks, recent)
        moved += len(a)
        want_w[0, h, b], want_p[0, h, b] = w0[0, h, a], p0[0, h, a]
        at = [torch.from_numpy(x).cuda() for x in (table_host[b // P].astype(np.int64), b % P, table_host[a // P].astype(np.int64),
                                                   a % P)]
        for t in want:
            t[at[0], at[1], h] = t[at[2], at[3], h]
    assert moved > 0
    assert (lens if in_place else kw["seq_lens_out"]).tolist() == [budget]
    assert np.array_equal(got_p.cpu().numpy(), want_p)
    assert np.array_equal(got_w.cpu().numpy(), want_w)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("budget,sinks,recent,ties,in_place", [
    (399000, 4, 1000, 0, True), (150000, 0, 0, 0, False), (30000, 7, 20000, 2, True), (399990, 0, 0, 3, False)])
def test_one_head_past_the_shared_keys_of_a_cluster(budget, sinks, recent, ties, in_place):
    # 400,001 tokens of one head over eight blocks: 50,016 keys each, 49,152 of which fit
    need_gpu()
    evict_long(400001, 1, 64, budget, sinks, recent, ties, in_place)


@pytest.mark.parametrize("drop,ties,in_place", [(10, 0, False), (16, 2, True), (500, 0, True), (20000, 1, False)])
def test_heads_past_the_shared_keys_of_a_block(drop, ties, in_place):
    # 150 heads fill the machine, a block each: 49,300 tokens, 49,152 of whose keys fit
    need_gpu()
    evict_long(49300, 150, 16, 49300 - drop, 4, 100, ties, in_place)


def test_window_over_an_evicted_cache_counts_indices():
    """window and sinks go by a token's index in the cache, whatever eviction left there; without them the order of
    a head's tokens does not matter."""
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    L, H, P, budget = 200, 2, 16, 120
    st = Streams([L], H, P, seed=31)
    rng = np.random.default_rng(5)
    w0 = rng.exponential(size=(1, H, st.cap)).astype(np.float32)
    p0 = np.tile(np.arange(st.cap, dtype=np.int32), (1, H, 1))
    w, p = torch.from_numpy(w0).cuda(), torch.from_numpy(p0).cuda()
    nxt, lens = st.lens_dev.clone(), st.lens_dev.clone()
    rkv.kvcache_paged_evict(st.cache, lens, w, p, nxt, budget, 4, 30)
    hk, hv = st.k[0][:budget].copy(), st.v[0][:budget].copy()
    for h in range(H):
        for a, b in evict_moves(w0[0, h, :L], p0[0, h, :L], L, budget, 4, 30):
            hk[b, h], hv[b, h] = st.k[0][a, h], st.v[0][a, h]
    pos = p[0, :, :budget].cpu().numpy()
    assert any(np.any(np.diff(pos[h]) < 0) for h in range(H))         # the newest are not the last any more
    st.lens, st.k, st.v = [budget], [hk], [hv]
    q = bf16_normal_bits(9, (1, 2 * H, D))
    scale = 1 / math.sqrt(D)
    for window, sinks in ((0, 0), (30, 4), (1, 0)):
        o = rkv.attn_decode_paged(to_dev(q), st.cache, lens, window=window, sinks=sinks)
        check_decode(st, q, o, scale, window, sinks)
    # each head's tokens by position: the same attention
    order = np.argsort(pos, axis=1)
    for h in range(H):
        hk[:, h], hv[:, h] = hk[order[h], h], hv[order[h], h]
    check_decode(st, q, rkv.attn_decode_paged(to_dev(q), st.cache, lens), scale)
