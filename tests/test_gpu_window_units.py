"""attn_fwd_window launches of more units than a schedule lists: the pairs of
SMs take them in turn."""

import pytest

from tests.test_gpu_window import run, spec

pytestmark = pytest.mark.gpu


def test_more_units_than_a_schedule_lists():
    run([spec(5, 130, 125, 40, 2)], 3970, 1, (1, 1))
    run([spec(3, 140, 100, 30, 1, seed=60), spec(2, 300, 298, 150, 0, seed=70)], 2000, 1, (1, 1))
    run([spec(2, 48, 1, 1, 1, 1, (True, True))], 3970, 1, (4, 6))
