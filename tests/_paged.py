"""A paged cache on the GPU beside its streams on the host, for the tests of
the paged calls."""

import numpy as np
import torch

from oracle import bf16_bits_to_f64, decode_ref, received_weight
from rolling_kv_cache_rope_b200.synth import bf16_normal_bits
from tests._gpu import to_dev, to_f64

D = 128
NAN = 0x7FC0   # a bf16 NaN: what unused rows of the pool hold


class Streams:
    """Streams of the given lengths in pages of P tokens, pages in random order
    in a pool with some to spare.  Every row outside a stream is NaN."""

    def __init__(self, lens, H, P, seed=0, spare=3, cols=None, interleaved=False, table_pad=0):
        from rolling_kv_cache_rope_b200 import rkv
        self.lens, self.H, self.P = list(lens), H, P
        n = len(lens)
        need = [-(-L // P) for L in lens]
        self.cols = max(1, max(need)) if cols is None else cols
        rng = np.random.default_rng(seed)
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages)
        self.table = np.full((n, self.cols + table_pad), -7, dtype=np.int32)   # unused entries: no page at all
        self.k = [bf16_normal_bits(seed + 10 * s + 1, (L, H, D)) for s, L in enumerate(lens)]
        self.v = [bf16_normal_bits(seed + 10 * s + 2, (L, H, D)) for s, L in enumerate(lens)]
        pool = np.full((n_pages, 2, P, H, D), NAN, dtype=np.uint16)
        at = 0
        for s, L in enumerate(lens):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
            for c in range(need[s]):
                m = min(P, L - c * P)
                pool[self.table[s, c], 0, :m] = self.k[s][c * P:c * P + m]
                pool[self.table[s, c], 1, :m] = self.v[s][c * P:c * P + m]
        if interleaved:
            both = to_dev(pool)
            kd, vd = both[:, 0], both[:, 1]
        else:
            kd, vd = to_dev(pool[:, 0]), to_dev(pool[:, 1])
        table = torch.from_numpy(self.table).cuda()[:, :self.cols]
        self.cache = rkv.PagedKVCache(kd, vd, table)
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    @property
    def n(self):
        return len(self.lens)

    @property
    def cap(self):
        return self.cols * self.P

    def rows(self, s):
        """(page, token in page) of each token of stream s."""
        j = np.arange(self.lens[s])
        return self.table[s, j // self.P], j % self.P

    def gathered(self, s):
        """bf16 bits of stream s as the pool holds them now."""
        pg, tk = (torch.from_numpy(np.ascontiguousarray(x)).long().cuda() for x in self.rows(s))
        f = lambda t: t[pg, tk].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        return f(self.cache.k), f(self.cache.v)


def decode_bounds(q, k, v, p, o, scale, H):
    """Largest error of o and of the received weight that the kernel's rounding
    allows, per value, from the oracle's own terms.

    Scores: 128 exact products in fp32, each of the 128 additions off by at
    most 2^-23 of the running sum of magnitudes (truncating adder); scale and
    exp2's argument add less than 2^-22 of the score, exp2 itself 2^-22.
    d = the largest relative error of a softmax term; numerator and sum each
    carry it.  P is rounded to bf16 for its product with V: 2^-8 (half a step)
    of each term; the sums over keys stay in fp32 (2^-23 per addition, at most
    the number of visible keys).  The output is rounded to bf16: 2^-8 of it."""
    Lq, Hq, L = p.shape
    G = Hq // H
    size = np.zeros((Lq, Hq))
    av = np.zeros_like(o)
    for h in range(Hq):
        size[:, h] = (np.abs(q[:, h]) @ np.abs(k[:, h // G]).T).max(1, initial=0.0) * scale if L else 0.0
        av[:, h] = p[:, h] @ np.abs(v[:, h // G]) if L else 0.0
    d = 2 * (128 * 2.0 ** -23 * size + 2.0 ** -20 + L * 2.0 ** -23)[:, :, None]
    o_err = (2.0 ** -8 + d) * av * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o) + 1e-30
    w_err = received_weight(p * d, H)
    return o_err, w_err


def check_decode(st, q_bits, o, scale, window=0, sinks=0, w_before=None, w_after=None):
    """o [n*Lq, Hq, D] (bf16 on the GPU) against the oracle; with w_before /
    w_after (fp32 numpy [n, H, cap]) the weights too."""
    n, Lq = st.n, q_bits.shape[0] // st.n
    got = to_f64(o)
    qf = bf16_bits_to_f64(q_bits)
    for s in range(n):
        q = qf[s * Lq:(s + 1) * Lq]
        k, v = bf16_bits_to_f64(st.k[s]), bf16_bits_to_f64(st.v[s])
        want, p = decode_ref(q, k, v, scale, window, sinks)
        o_err, w_err = decode_bounds(q, k, v, p, want, scale, st.H)
        off = np.abs(got[s * Lq:(s + 1) * Lq] - want)
        assert np.all(off <= o_err), (s, float((off - o_err).max()), float(off.max()))
        if w_after is None:
            continue
        L = st.lens[s]
        before = w_before[s, :, :L].astype(np.float64) if w_before is not None else np.zeros((st.H, L))
        add = received_weight(p, st.H)
        lim = w_err + 2.0 ** -23 * (np.abs(before) + add) + 1e-30
        off = np.abs(w_after[s, :, :L] - (before + add))
        assert np.all(off <= lim), (s, float((off - lim).max()))
