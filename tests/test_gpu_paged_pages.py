"""Tokens on pages outside the pool: a call leaves out the whole token, its row
and its scores, and everything else is as without it."""

import numpy as np
import pytest
import torch

from oracle import evict_moves
from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import need_gpu, to_dev
from tests._paged import D, Streams

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


# (lens, H, P, budget, columns of the page table of the first stream that are no page): the survivors
# and the places that fall free lie on good and on bad pages; few tokens to drop, many, many over a cluster
EVICTIONS = [
    ([64, 50], 2, 4, 54, (14, 2)),
    ([64, 50], 2, 4, 54, (15,)),
    ([64, 50], 2, 4, 54, (0, 1, 5)),
    ([300, 280], 3, 16, 200, (15, 3, 7)),
    ([6000], 1, 16, 2500, (200, 3, 370, 80)),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,H,P,budget,bad", EVICTIONS)
def test_evict_moves_rows_and_scores_together(lens, H, P, budget, bad, in_place):
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams(lens, H, P, seed=21)
    n, cap = st.n, st.cap
    rng = np.random.default_rng(budget + len(bad))
    w0 = rng.exponential(size=(n, H, cap)).astype(np.float32)
    p0 = np.stack([np.stack([rng.permutation(cap) for _ in range(H)]) for _ in range(n)]).astype(np.int32)
    pages = st.cache.k.shape[0]
    for i, col in enumerate(bad):
        st.cache.page_table[0, col] = (-1, pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    w, p, lens_in = torch.from_numpy(w0).cuda(), torch.from_numpy(p0).cuda(), st.lens_dev.clone()
    nxt = torch.full((n,), cap, dtype=torch.int32, device="cuda")
    k0, v0 = bits(st.cache.k).clone(), bits(st.cache.v).clone()
    kw = {} if in_place else dict(seq_lens_out=torch.zeros_like(lens_in), weight_out=torch.full_like(w, 5.0),
                                  pos_out=torch.full_like(p, 5))
    rkv.kvcache_paged_evict(st.cache, lens_in, w, p, nxt, budget, 2, 5, **kw)
    with pytest.raises(rkv.RkvError, match="page"):
        rkv.rkv_paged_status(st.cache)
    want_w, want_p = (w0.copy(), p0.copy()) if in_place else (np.full_like(w0, 5.0), np.full_like(p0, 5))
    done = left = 0
    for s, L in enumerate(lens):
        m = min(L, budget)
        want_w[s, :, :m], want_p[s, :, :m] = w0[s, :, :m], p0[s, :, :m]
        pg, tk = st.rows(s)
        for h in range(H):
            for a, b in evict_moves(w0[s, h, :L], p0[s, h, :L], cap, budget, 2, 5):
                if s == 0 and (a // P in bad or b // P in bad):
                    left += 1
                    continue
                done += 1
                want_w[s, h, b], want_p[s, h, b] = w0[s, h, a], p0[s, h, a]
                k0[pg[b], tk[b], h], v0[pg[b], tk[b], h] = k0[pg[a], tk[a], h], v0[pg[a], tk[a], h]
    assert done > 0 and left > 0
    got_lens, got_w, got_p = (lens_in, w, p) if in_place else (kw["seq_lens_out"], kw["weight_out"], kw["pos_out"])
    assert got_lens.tolist() == [min(L, budget) for L in lens]
    assert torch.equal(bits(st.cache.k), k0) and torch.equal(bits(st.cache.v), v0)
    assert np.array_equal(got_p.cpu().numpy(), want_p)
    assert np.array_equal(got_w.cpu().numpy(), want_w)


@pytest.mark.parametrize("lens,H,P,new", [([40, 9], 2, 16, 1), ([40, 9], 3, 4, 12), ([500], 12, 16, 33)])
def test_insert_leaves_scores_of_tokens_without_a_page(lens, H, P, new):
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    st = Streams(lens, H, P, seed=22)
    n, L = st.n, lens[0]
    bad = (L - 1) // P            # the page of the first stream's newest token
    st.cache.page_table[0, bad] = st.cache.k.shape[0]
    kb, vb = bf16_normal_bits(50, (n * new, H, D)), bf16_normal_bits(51, (n * new, H, D))
    k0, v0 = bits(st.cache.k).clone(), bits(st.cache.v).clone()
    pos = torch.full((n, H, st.cap), -1, dtype=torch.int32, device="cuda")
    weight = torch.full((n, H, st.cap), 2.5, device="cuda")
    rkv.kvcache_paged_insert(st.cache, to_dev(kb), to_dev(vb), st.lens_dev, next_pos=st.lens_dev + 500, pos=pos, weight=weight)
    with pytest.raises(rkv.RkvError, match="page"):
        rkv.rkv_paged_status(st.cache)
    want_p, want_w = np.full(pos.shape, -1), np.full(weight.shape, 2.5)
    for s, x in enumerate(lens):
        pg, tk = st.rows(s)
        for i in range(new):
            j = x - new + i
            if j < 0 or (s == 0 and j // P == bad):
                continue
            for t, src in ((k0, kb), (v0, vb)):
                t[pg[j], tk[j]] = torch.from_numpy(src[s * new + i].view(np.int16)).cuda()
            want_p[s, :, j], want_w[s, :, j] = x + 500 - new + i, 0.0
    assert torch.equal(bits(st.cache.k), k0) and torch.equal(bits(st.cache.v), v0)
    assert np.array_equal(pos.cpu().numpy(), want_p)
    assert np.array_equal(weight.cpu().numpy(), want_w)
