"""Pins of the paged-cache oracle and of the windowed mask: hand tables, the
plain attention oracle, torch's float64 SDPA, properties of the eviction."""

import numpy as np
import pytest
import torch

from oracle import (attention_ref, decode_ref, evict_moves, frame_block_visible, frame_window_visible, received_weight,
                    token_visible)


def test_token_visible_hand_table():
    # 6 tokens, the newest two ask, each sees two tokens and the first one
    want = np.array([[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]], dtype=bool)
    assert np.array_equal(token_visible(6, 2, 2, 1), want)
    # more queries than tokens: the first ones lie before the stream
    assert np.array_equal(token_visible(1, 3, 0, 0), np.array([[0], [0], [1]], dtype=bool))
    assert token_visible(0, 2, 0, 0).shape == (2, 0)


def test_frame_window_visible_hand_table():
    # frames of 2 tokens, blocks of 1 frame, 4 frames; queries are frames 2 and 3; window 2, one sink
    got = frame_window_visible(4, 8, 2, 2, 1, 2, 1)
    f2 = [1, 1, 1, 1, 1, 1, 0, 0]
    f3 = [1, 1, 0, 0, 1, 1, 1, 1]
    assert np.array_equal(got, np.array([f2, f2, f3, f3], dtype=bool))
    # no window: the block mask
    assert np.array_equal(frame_window_visible(30, 70, 5, 3, 2, 0, 1), frame_block_visible(30, 70, 5, 3, 2))
    # sinks never reach past the query's own block
    assert not frame_window_visible(2, 20, 2, 0, 1, 1, 9)[:, 2:].any()


@pytest.mark.parametrize("L,Lq,H,G,window,sinks", [(9, 1, 2, 1, 0, 0), (9, 3, 1, 2, 4, 1), (2, 4, 1, 1, 0, 0)])
def test_decode_ref_is_masked_attention(L, Lq, H, G, window, sinks):
    rng = np.random.default_rng(L + Lq)
    q, k, v = rng.standard_normal((Lq, H * G, 8)), rng.standard_normal((L, H, 8)), rng.standard_normal((L, H, 8))
    o, p = decode_ref(q, k, v, 0.3, window, sinks)
    kk, vv = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    seen = token_visible(L, Lq, window, sinks)
    assert np.allclose(o, attention_ref(q, kk, vv, 0.3, seen), atol=1e-13)
    rows = seen.any(1)
    if rows.any():
        t = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q[rows]).transpose(0, 1), torch.tensor(kk).transpose(0, 1), torch.tensor(vv).transpose(0, 1),
            attn_mask=torch.tensor(seen[rows]), scale=0.3).transpose(0, 1).numpy()
        assert np.allclose(o[rows], t, atol=1e-13)
    assert np.allclose(p.sum(-1), np.repeat(rows[:, None], H * G, 1))
    w = received_weight(p, H)
    assert w.shape == (H, L) and np.isclose(w.sum(), rows.sum() * H * G)
    assert np.allclose(w[0], p[:, :G].sum((0, 1)))


def test_evict_moves_by_hand():
    # 7 tokens to 4: token 0 is a sink, 6 the newest; of the others 5 and 3 weigh most
    w, pos = [0.0, 1.0, 0.5, 3.0, 0.1, 2.0, 0.0], list(range(7))
    assert evict_moves(w, pos, 7, 4, 1, 1) == [(5, 1), (6, 2)]
    # ties go to the lowest index, NaN below every number
    assert evict_moves([1.0, 1.0, 1.0, 1.0], [5, 6, 7, 8], 9, 2, 0, 0) == []
    assert evict_moves([np.nan, -np.inf, 1.0], [5, 6, 7], 9, 2, 0, 0) == [(2, 0)]
    assert evict_moves([0.0, -0.0, 0.0], [5, 6, 7], 9, 2, 0, 0) == []
    assert evict_moves([1.0], [0], 1, 1, 0, 0) == []


def test_evict_keeps_the_heaviest():
    rng = np.random.default_rng(0)
    for _ in range(50):
        L, B = int(rng.integers(1, 40)), int(rng.integers(1, 40))
        w, pos = rng.integers(0, 6, L).astype(float), rng.permutation(L)
        sinks, recent = int(rng.integers(0, B + 1)), 0
        moves = evict_moves(w, pos, L, B, sinks, recent)
        state = list(range(L))
        for a, b in moves:
            assert a >= B > b
            state[b] = a
        kept = state[:min(B, L)]
        assert len(set(kept)) == len(kept)
        guard = [j for j in range(L) if pos[j] < sinks]
        assert set(guard) <= set(kept)
        free = sorted((w[j] for j in range(L) if j not in guard), reverse=True)[:len(kept) - len(guard)]
        assert sorted((w[j] for j in kept if j not in guard), reverse=True) == free
