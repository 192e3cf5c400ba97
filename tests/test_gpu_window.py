"""attn_fwd_window on the GPU against the float64 oracle."""

import math

import numpy as np
import pytest
import torch

from oracle import attention_ref, bf16_bits_to_f64, frame_window_visible, rope3d_ref
from rolling_kv_cache_rope_b200.synth import DENOISE, bf16_normal_bits
from tests._gpu import ATTN_REL_L2, need_gpu, to_dev, to_f64

pytestmark = pytest.mark.gpu
D = 128
SCALE = 1.0 / math.sqrt(D)


def bound(q, k, v, seen, o, rope_q, rope_k):
    """Largest error per output that the kernel's rounding allows: scores off by
    128 fp32 additions (2^-23 each of the sum of magnitudes) and, where Q or K
    is rotated in the kernel, by its rounding to bf16 (2^-8 of each value, plus
    2^-20 for the fp32 rotation); the softmax terms carry e^(2d) - 1 of that;
    P rounded to bf16 (2^-8), fp32 sums, the output rounded to bf16 (2^-8)."""
    av = np.zeros_like(o)
    G = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        kh, vh = k[:, h // G], np.abs(v[:, h // G])
        s = np.where(seen, (q[:, h] @ kh.T) * SCALE, -np.inf)
        m = s.max(1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(m), m, 0))
        l = p.sum(1, keepdims=True)
        p = np.where(l > 0, p / np.where(l > 0, l, 1), 0)
        mag = (np.abs(q[:, h]) @ np.abs(kh).T) * SCALE
        # rotation mixes two values: magnitudes of a rotated pair grow by sqrt(2) at most
        per = 128 * 2.0 ** -23 + ((2.0 ** -8 + 2.0 ** -20) * 1.5) * (int(rope_q) + int(rope_k))
        d = (mag * per * (p > 0)).max(1, keepdims=True)
        av[:, h] = (np.exp(2 * d) - 1 + 2.0 ** -8 + 2.0 ** -16) * (p @ vh)
    return av * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o) + 1e-30


def run(specs, H, G, grid, layout="adjacent", pairs=(22, 21, 21), poison=True, strided=False, rows=None):
    """specs: Lq, Lk, off, block, window, sinks, rope (q, k), seed.  One launch."""
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    F = grid[0] * grid[1]
    seqs, wins, host = [], [], []
    for sp in specs:
        Lq, Lk = sp["Lq"], sp["Lk"]
        qb = bf16_normal_bits(sp["seed"], (Lq, H * G, D))
        kb, vb = bf16_normal_bits(sp["seed"] + 1, (Lk, H, D)), bf16_normal_bits(sp["seed"] + 2, (Lk, H, D))
        seen = frame_window_visible(Lq, Lk, F, sp["off"], sp["block"], sp["window"], sp["sinks"], rows=rows)
        if poison and rows is None:     # keys no row sees hold NaN and infinities
            dead = ~seen.any(0)
            kb[dead], vb[dead] = 0x7FC0, 0x7F80
        q, k, v = to_dev(qb), to_dev(kb), to_dev(vb)
        if strided:
            wide = torch.zeros(Lk, 2 * H + 1, D, dtype=torch.bfloat16, device="cuda")
            wide[:, :H], wide[:, H + 1:] = k, v
            k, v = wide[:, :H], wide[:, H + 1:]
        out = torch.full((Lq + 2, H * G + 1, D), -3.0, dtype=torch.bfloat16, device="cuda")
        o = out[1:-1, 1:]
        seqs.append(rkv.AttnSeq(q, k, v, o, q_t0=sp["off"], k_t0=0, rope_q=sp["rope"][0], rope_k=sp["rope"][1],
                                block_frames=sp["block"], q_frame_offset=sp["off"]))
        wins.append((sp["window"], sp["sinks"]))
        host.append((qb, kb, vb, seen, out))
    ws = rkv.attn_fwd_window(seqs, wins, rkv.make_rope(*grid, pairs, layout=layout))
    rkv.rkv_attn_status(ws)
    torch.cuda.synchronize()
    for sp, (qb, kb, vb, seen, out) in zip(specs, host):
        take = np.arange(sp["Lq"]) if rows is None else rows
        q, k, v = bf16_bits_to_f64(qb)[take], bf16_bits_to_f64(kb), bf16_bits_to_f64(vb)
        dead = ~seen.any(0)
        k[dead], v[dead] = 0.0, 0.0
        if sp["rope"][0]:
            q = rope3d_ref(q, sp["off"], *grid, pairs, token_index=take, layout=layout)
        if sp["rope"][1]:
            k = rope3d_ref(k, 0, *grid, pairs, layout=layout)
        want = attention_ref(q, np.repeat(k, G, 1), np.repeat(v, G, 1), SCALE, seen)
        got = to_f64(out)[1:-1, 1:][take]
        off = np.abs(got - want)
        lim = bound(q, k, v, seen, want, *sp["rope"])
        assert np.all(off <= lim), (sp, float((off - lim).max()), float(off.max()))
        assert np.linalg.norm(got - want) <= ATTN_REL_L2 * max(np.linalg.norm(want), 1e-30), sp
        empty = ~seen.any(1)
        assert np.all(got[empty] == 0.0)
        assert torch.all(out[0] == -3.0) and torch.all(out[-1] == -3.0) and torch.all(out[:, 0] == -3.0)


def spec(Lq, Lk, off, window, sinks, block=1, rope=(False, False), seed=40):
    return dict(Lq=Lq, Lk=Lk, off=off, window=window, sinks=sinks, block=block, rope=rope, seed=seed)


@pytest.mark.parametrize("Lq,Lk,off,window,sinks,block", [
    (1, 1, 0, 1, 0, 1),
    (1, 700, 699, 100, 4, 1),
    (1, 700, 699, 1, 0, 1),
    (65, 65, 0, 3, 1, 1),
    (700, 700, 0, 100, 4, 1),
    (700, 700, 0, 0, 0, 1),                  # causal, no window
    (513, 1400, 887, 200, 130, 1),           # sinks past a tile
    (1100, 1100, 0, 30, 0, 1),               # windows shorter than a tile
    (1100, 1100, 0, 129, 1, 1),
    (600, 40, 0, 3, 0, 1),                   # queries past the keys: rows that see nothing
    (600, 40, 100, 3, 0, 1),                 # no row sees a key
    (600, 40, 100, 3, 2, 1),                 # only the sinks
    (300, 1000, 40, 4, 2, 16),
    (1537, 1537, 0, 2, 3, 50),
])
def test_token_windows(Lq, Lk, off, window, sinks, block):
    run([spec(Lq, Lk, off, window, sinks, block)], 1, 2, (1, 1))


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 4), (1, 7)])
def test_grouped_heads(H, G):
    run([spec(300, 420, 120, 150, 10)], H, G, (1, 1))


@pytest.mark.parametrize("H,G", [(2, 1), (3, 2), (2, 4), (1, 8)])
def test_split_units(H, G):
    # few units of many key tiles run as several parts, merged into the output
    run([spec(900, 2500, 1600, 1300, 140)], H, G, (1, 1))
    run([spec(70, 6001, 5931, 5000, 3)], H, G, (1, 1), rows=np.r_[0:3, 40, 67:70])
    # rows whose window some parts miss altogether
    run([spec(520, 3000, 2480, 900, 0)], H, G, (1, 1), rows=np.r_[0:4, 127:130, 510:520])


def test_windows_with_rope_and_grouped_heads():
    run([spec(500, 720, 10, 3, 1, 1, (True, True))], 2, 4, (4, 6))
    run([spec(500, 720, 10, 3, 1, 1, (True, True))], 2, 2, (4, 6))


def test_small_workspace():
    # with room for the status word only nothing is split: the same result within rounding
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    q, k, v = (to_dev(bf16_normal_bits(30 + i, (n, 2, D))) for i, n in enumerate((700, 2000, 2000)))
    outs = []
    for ws in (None, torch.empty(256, dtype=torch.uint8, device="cuda")):
        o = torch.full_like(q, float("nan"))
        s = rkv.AttnSeq(q, k, v, o, rope_q=False, rope_k=False, block_frames=1, q_frame_offset=1300)
        rkv.rkv_attn_status(rkv.attn_fwd_window([s], [(1000, 3)], rkv.make_rope(1, 1), workspace=ws))
        outs.append(to_f64(o))
    # both round P and the output to bf16: half a step each of the weights' and of the output's size
    assert np.abs(outs[0] - outs[1]).max() <= 4 * 2.0 ** -8 * np.abs(outs[0]).max()


@pytest.mark.parametrize("rope", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("Lq,Lk,off,window,sinks,block", [
    (72, 120, 2, 2, 1, 1), (100, 121, 1, 1, 1, 3), (600, 960, 15, 6, 2, 1), (600, 960, 15, 2, 1, 3)])
def test_frame_windows_with_rope(Lq, Lk, off, window, sinks, block, rope):
    run([spec(Lq, Lk, off, window, sinks, block, rope)], 2, 1, (4, 6))


def test_rope_variants():
    run([spec(150, 240, 3, 2, 1, 1, (True, True))], 2, 2, (4, 6), layout="half")
    run([spec(150, 240, 3, 2, 1, 1, (True, True))], 2, 2, (4, 6), pairs=(30, 18, 16))


def test_sequences_of_one_launch():
    run([spec(300, 300, 0, 40, 1, seed=60), spec(1, 900, 899, 128, 0, seed=70), spec(700, 800, 100, 0, 0, seed=80),
         spec(20, 500, 480, 600, 3, seed=90)], 2, 2, (1, 1))


def test_strided_keys():
    run([spec(200, 260, 60, 70, 5)], 2, 2, (1, 1), strided=True)


def test_equal_units_with_tail_split():
    # every unit sees the same number of tiles, and the last wave of units is short: 16 heads x 10 blocks
    rows = np.unique(np.r_[0:5, 505:520, 2555:2565, 5115:5120])
    run([spec(5120, 6400, 1280, 1280, 0, 1280)], 16, 1, (1, 1), rows=rows)


def test_no_window_is_the_block_mask():
    # bit-identical to attn_fwd_varlen where the mask and the heads are the same (and the workspace
    # leaves no room to split units, which joins two halves' sums in another order)
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    q, k, v = (to_dev(bf16_normal_bits(20 + i, (n, 2, D))) for i, n in enumerate((480, 720, 720)))
    rope = rkv.make_rope(4, 6)
    outs = []
    for window in (None, 0, 1000):
        o = torch.full_like(q, float("nan"))
        s = rkv.AttnSeq(q, k, v, o, q_t0=10, k_t0=0, block_frames=3, q_frame_offset=10)
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        if window is None:
            rkv.attn_fwd_varlen([s], rope, workspace=ws)
        else:
            rkv.attn_fwd_window([s], [(window, 0)], rope, workspace=ws)
        rkv.rkv_attn_status(ws)
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_full_size_sampled():
    F = DENOISE.frame_tokens
    rng = np.random.default_rng(0)
    rows = {0, 1, DENOISE.Lq - 1}
    for f in range(1, DENOISE.q_frames):
        rows |= {f * F - 1, f * F}
    rows |= set(int(x) for x in rng.integers(0, DENOISE.Lq, 12))
    run([spec(DENOISE.Lq, DENOISE.Lk, DENOISE.q_t0, 4, 1, 3, (True, True))], 12, 1, (30, 52),
        rows=np.array(sorted(rows)))


def test_many_tokens_no_table():
    # a frame grid too large for the rotation table is fine where nothing is rotated
    run([spec(90, 90, 0, 1, 0)], 1, 1, (400, 300))


def test_other_stream_and_captured():
    need_gpu()
    from rolling_kv_cache_rope_b200 import rkv
    q, k, v = (to_dev(bf16_normal_bits(30 + i, (333, h, D))) for i, h in enumerate((4, 2, 2)))
    rope = rkv.make_rope(1, 1)
    o = torch.empty_like(q)

    def call(out, **kw):
        s = rkv.AttnSeq(q, k, v, out, rope_q=False, rope_k=False, block_frames=1)
        return rkv.attn_fwd_window([s], [(64, 2)], rope, **kw)

    rkv.rkv_attn_status(call(o))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = torch.zeros_like(q)
    side.wait_stream(torch.cuda.current_stream())
    ws = call(o2, stream=side)
    side.synchronize()
    assert torch.equal(o, o2)
    o3 = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(o3, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o3)


@pytest.mark.parametrize("off,block,window,sinks", [
    (2 ** 31 - 1000, 1, 50, 3), (2 ** 31 - 1000, 7, 50, 0), (0, 2 ** 31 - 1, 1, 0), (100, 1, 2 ** 31 - 1, 0),
    (100, 3, 2, 2 ** 31 - 1), (2 ** 31 - 1000, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1),
])
def test_masks_at_their_largest(off, block, window, sinks):
    run([spec(200, 300, off, window, sinks, block)], 1, 2, (1, 1))
