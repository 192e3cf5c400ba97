"""attn_decode_paged with more than 64 query rows to a key head: several row
blocks, the last partly filled, over several key heads, items that end whole in
one block of the launch and items that go on in others."""

import numpy as np
import pytest
import torch

from tests._gpu import need_gpu
from tests._paged import Streams, check_decode
from tests.test_gpu_paged_decode import SCALE, queries, run

pytestmark = pytest.mark.gpu
SHORT = [int(x) for x in np.random.default_rng(4).integers(0, 50, 220)]

CASES = [
    # lens, H, G, P, Lq, window, sinks
    ([300, 9, 40], 2, 10, 16, 7, 0, 0),        # 70 rows: the second block has 6
    ([5000], 3, 13, 64, 5, 0, 0),              # 65: the second block has 1
    ([700, 33], 2, 127, 16, 1, 0, 0),          # 127
    ([90, 800, 0], 1, 43, 16, 3, 0, 0),        # 129: three blocks
    (SHORT, 2, 35, 16, 2, 0, 0),               # items of one step, several to a block of the launch
    ([700, 20, 1300], 3, 24, 13, 3, 200, 9),   # 72, a window that starts inside pages
    ([2, 64, 500], 2, 70, 16, 4, 5, 0),        # 280 rows, windows that end between the queries
]


@pytest.mark.parametrize("lens,H,G,P,Lq,window,sinks", CASES)
def test_row_blocks(lens, H, G, P, Lq, window, sinks):
    need_gpu()
    st = Streams(lens, H, P, seed=13)
    q = queries(st, Lq, G)
    kw = dict(window=window, sinks=sinks)
    o = run(st, q, **kw)
    check_decode(st, q, o, SCALE, window, sinks)
    before = torch.rand(st.n, H, st.cap, device="cuda")
    after = torch.full_like(before, -5.0)
    with_weights = run(st, q, weight_in=before, weight_out=after, **kw)
    assert torch.equal(with_weights, o)
    check_decode(st, q, o, SCALE, window, sinks, before.cpu().numpy(), after.cpu().numpy())
    for s, L in enumerate(lens):
        assert torch.all(after[s, :, L:] == -5.0)
