"""Paged cache operators at the ends of their arguments' ranges (B200 only)."""
import math

import pytest
import torch

from tests import paged_ref as R
from tests.test_gpu_paged import BF, DEV, HF, SHARED, _gen, check_rows, host, ints, make_kv, make_pool, make_tables, \
    run_attn, whole

pytestmark = pytest.mark.gpu

LOW = -2 ** 31


# ------------------------------------------------------------------ row limits
@pytest.mark.parametrize("case", [
    (BF, 128, 28, 4, 16, "heads", [4, 2], whole(300, 1000)),            # 32-row tiles
    (HF, 64, 8, 2, 64, "slots", [70, 33], whole(700, 390)),             # 128-row tiles
    (BF, 32, 4, 4, 8, "padded", [3], [((130, 70), (260, 300))]),
], ids=lambda c: str(c)[:60])
@pytest.mark.parametrize("low", [LOW, LOW + 1, LOW + 127, LOW + 300])
def test_lowest_row_limits_see_nothing(case, low):
    """Rows whose limit is at the low end of int32, beside rows that keep every key tile alive."""
    f = lambda s, j: 2 ** 31 - 1 if j % 2 else low  # noqa: E731
    run_attn(*case, limit=f)
    n = len(case[6])
    run_attn(*case, limit=f, groups=([0, n], [140]))
    run_attn(*case, limit=f, groups=([0, n], [0]))


def test_lowest_row_limits_beside_other_sequences():
    for c in (SHARED[1], SHARED[5], SHARED[8]):
        run_attn(*c[:8], groups=c[8], limit=lambda s, j: LOW if s % 2 else 2 ** 31 - 1)
