"""attn_fwd_window's mask and key-tile plan, evaluated on the host by the
kernel's own functions, against the mask oracle; and its refusals (no GPU)."""

import ctypes

import numpy as np
import pytest

from oracle import frame_window_visible


@pytest.fixture(scope="module")
def rkv(lib_path):
    from rolling_kv_cache_rope_b200 import rkv as m
    return m


def check(rkv, grid, seqs, windows, H=2, H_kv=2):
    F = grid[0] * grid[1]
    sink, begin, limit, units = rkv.attn_window_rows(seqs, windows, H, rkv.make_rope(*grid), H_kv)
    G = H // H_kv
    pack = 4 if G % 4 == 0 else 2 if G % 2 == 0 else 1
    rows = 512 // pack
    want_units = sorted((i, h, r) for i, s in enumerate(seqs) for h in range(0, H, pack) for r in range(0, s["Lq"], rows))
    assert sorted(map(tuple, units[:, :3].tolist())) == want_units
    for i, (s, (w, k)) in enumerate(zip(seqs, windows)):
        Lq, Lk = s["Lq"], s["Lk"]
        seen = frame_window_visible(Lq, Lk, F, s.get("q_frame_offset", 0), s["block_frames"], w, k)
        c = np.arange(Lk)[None, :]
        got = (c < limit[i][:, None]) & ((c >= begin[i][:, None]) | (c < sink[i][:, None]))
        assert np.array_equal(got, seen), (s, w, k)
        # a unit's tiles: every tile that holds a key one of its rows sees, or one tile; a tile between
        # the sinks and the window may be taken in where the two runs meet
        for si, head, row0, tiles in units:
            if si != i:
                continue
            last = min(Lq, row0 + rows) - 1
            pad = np.zeros(-(-Lk // 128) * 128, dtype=bool)
            pad[:Lk] = seen[row0:last + 1].any(0)
            need = pad.reshape(-1, 128).any(1)
            assert need.sum() <= tiles, (s, w, k, row0, tiles)
            # never more than the span of the rows' windows and the sinks
            most = -(-int(limit[i][last]) // 128) - int(begin[i][row0]) // 128 + -(-int(sink[i].max()) // 128)
            assert tiles <= max(1, most), (s, w, k, row0, tiles, most)


@pytest.mark.parametrize("grid,Lq,Lk,off,block,window,sinks", [
    ((1, 1), 700, 700, 0, 1, 100, 4),
    ((1, 1), 1, 900, 899, 1, 128, 130),
    ((1, 1), 5, 900, 0, 1, 1, 0),
    ((1, 1), 600, 40, 0, 1, 3, 0),        # queries past the keys: rows that see nothing
    ((1, 1), 300, 40, 100, 16, 2, 1),
    ((4, 6), 100, 120, 0, 1, 2, 1),
    ((4, 6), 72, 121, 2, 3, 1, 0),
    ((15, 26), 1950, 2730, 2, 1, 3, 1),
    ((30, 52), 23400, 32760, 6, 3, 4, 1),
    ((30, 52), 1560, 32760, 20, 3, 0, 5),
])
def test_plan_matches_oracle(rkv, grid, Lq, Lk, off, block, window, sinks):
    for H, H_kv in ((2, 2), (4, 1), (6, 1), (6, 3)):
        check(rkv, grid, [dict(Lq=Lq, Lk=Lk, q_frame_offset=off, block_frames=block)], [(window, sinks)], H, H_kv)


def test_plan_random(rkv):
    rng = np.random.default_rng(3)
    for _ in range(40):
        grid = (int(rng.integers(1, 5)), int(rng.integers(1, 7)))
        seqs, windows = [], []
        for _ in range(int(rng.integers(1, 4))):
            seqs.append(dict(Lq=int(rng.integers(1, 1300)), Lk=int(rng.integers(1, 2000)),
                             q_frame_offset=int(rng.integers(0, 100)), block_frames=int(rng.integers(1, 4))))
            windows.append((int(rng.integers(0, 30)), int(rng.integers(0, 8))))
        G = int(rng.integers(1, 9))
        check(rkv, grid, seqs, windows, H=G, H_kv=1)


def desc(rkv, **kw):
    d = dict(q=0x100000, k=0x10000000, v=0x20000000, o=0x30000000, q_stride=512, k_stride=256, v_stride=256, o_stride=512,
             Lq=10, Lk=20, block_frames=1)
    d.update(kw)
    return rkv.rkv_attn_seq(**d)


@pytest.mark.parametrize("seq,win,call,frag", [
    (dict(block_frames=0), (1, 1), {}, "block_frames"),
    (dict(), (-1, 0), {}, "window_blocks"),
    (dict(), (0, -1), {}, "sink_blocks"),
    (dict(), (1, 0), dict(H_kv=3), "multiple"),
    (dict(), (1, 0), dict(H_kv=0), "multiple"),
    (dict(), None, {}, "windows"),
    (dict(k_stride=128), (1, 0), {}, "stride"),
    (dict(o=0x10000000), (1, 0), {}, "overlap"),
    (dict(q_frame_offset=-1), (1, 0), {}, "q_frame_offset"),
    (dict(), (1, 0), dict(D=64), "128"),
    (dict(), (1, 0), dict(ws=0), "workspace"),
])
def test_window_rejects(rkv, seq, win, call, frag):
    a = dict(H=4, H_kv=2, D=128, ws=0x40000000)
    a.update(call)
    s = desc(rkv, **seq)
    w = rkv.rkv_attn_window(*win) if win else None
    rope = rkv.make_rope(1, 1)
    st = rkv.lib().attn_fwd_window(ctypes.byref(s), ctypes.byref(w) if win else None, 1, a["H"], a["H_kv"], a["D"], 0.1,
                                   ctypes.byref(rope), ctypes.c_void_p(a["ws"]), 256, None)
    assert st == rkv.RKV_ERR_INVALID_ARG, rkv.rkv_last_error_string()
    assert frag in rkv.rkv_last_error_string()


def test_window_rejects_far_frames(rkv):
    s, w, rope = desc(rkv, q_frame_offset=2 ** 31 - 1), rkv.rkv_attn_window(1, 0), rkv.make_rope(1, 1)
    st = rkv.lib().attn_fwd_window(ctypes.byref(s), ctypes.byref(w), 1, 4, 2, 128, 0.1, ctypes.byref(rope),
                                   ctypes.c_void_p(0x40000000), 256, None)
    assert st == rkv.RKV_ERR_UNSUPPORTED and "frame" in rkv.rkv_last_error_string()


def test_window_rows_rejects(rkv):
    with pytest.raises(rkv.RkvError, match="block_frames"):
        rkv.attn_window_rows([dict(Lq=1, Lk=1, block_frames=0)], [(1, 1)], 1, rkv.make_rope(1, 1))
    with pytest.raises(rkv.RkvError, match="window_blocks"):
        rkv.attn_window_rows([dict(Lq=1, Lk=1, block_frames=1)], [(-2, 1)], 1, rkv.make_rope(1, 1))


@pytest.mark.parametrize("block,window,sinks", [(2 ** 30, 2 ** 31 - 1, 0), (2 ** 30, 2 ** 31 - 1, 2 ** 31 - 1),
                                                (1, 2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1, 4), (1, 2 ** 40 + 1, 2 ** 40)])
def test_window_past_everything(rkv, block, window, sinks):
    """Windows, blocks and sinks whose products pass 64 bits see all that the block mask leaves."""
    seqs = [dict(Lq=1000, Lk=9000, block_frames=block, q_frame_offset=3)]
    got = rkv.attn_window_rows(seqs, [(window, sinks)], 1, rkv.make_rope(30, 52))
    ref = rkv.attn_window_rows(seqs, [(0, 0)], 1, rkv.make_rope(30, 52))
    assert (np.asarray(got[1][0]) == 0).all()
    assert (np.asarray(got[2][0]) == np.asarray(ref[2][0])).all()


def test_sinks_past_64_bits(rkv):
    """2^14 first blocks of 2^30 frames of 2^20 tokens: every key up to the row's limit."""
    seqs = [dict(Lq=20, Lk=50000, block_frames=2 ** 30)]
    sink, _, limit, _ = rkv.attn_window_rows(seqs, [(1, 2 ** 14)], 1, rkv.make_rope(2 ** 10, 2 ** 10))
    assert (np.asarray(sink[0]) == 50000).all() and (np.asarray(limit[0]) == 50000).all()
