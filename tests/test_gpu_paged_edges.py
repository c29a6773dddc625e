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


# ------------------------------------------------------------------ queries that are not finite
@pytest.mark.parametrize("case", [
    (BF, 128, 28, 4, 16, "heads", [1, 3], whole(20, 100)),       # 32-row tiles, whole
    (HF, 64, 8, 2, 64, "slots", [40, 90], whole(100, 60)),       # 128-row tiles, whole
    (BF, 128, 28, 4, 16, "heads", [1], whole(40000)),            # 32-row tiles, cut over all CTAs
    (HF, 32, 4, 1, 64, "heads", [40], whole(30000)),             # 128-row tiles, cut
], ids=lambda c: str(c)[:60])
@pytest.mark.parametrize("grouped", [False, True])
def test_rows_that_are_not_numbers_stay_so(case, grouped):
    """A query of NaN, or infinities whose scores are none, gives NaN in its own row and head
    however its tile is cut; the other rows and heads are as ever, and a row without keys
    gives 0 whatever its query holds."""
    dtype, D, hq, hkv, ps, layout, rows, segs = case
    g = _gen(77)
    lens = [sg[0][1] for sg in segs]
    n_pages = sum(-(-n // ps) for n in lens) + 5
    pool = make_pool(g, n_pages, hkv, ps, D, dtype, layout)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, at = make_tables(lens, ps, order)
    ptable, _ = make_tables([50] if ps >= 16 else [20], ps, order, at)
    n, rs = sum(rows), [sum(rows[:i]) for i in range(len(rows) + 1)]
    q = torch.randn(n, hq, D, generator=g).to(dtype).to(DEV)
    kv = make_kv(pool, hq, n, 1)
    lim = [2 ** 31 - 1] * n
    if n > 1 and not grouped:
        lim[n - 1] = 0

    def call(x):
        out, lse = torch.full_like(q, 3.0), torch.full((n, hq), 5.0, device=DEV)
        a = (x, ints(rs), table.to(DEV), ints(segs))
        if grouped:
            kv.shared_prefix_attn(*a, ints([0, len(rows)]), ptable.to(DEV), ints([20]), out=out, lse=lse)
        else:
            kv.attn(*a, row_limit=ints(lim), out=out, lse=lse)
        return out, lse

    want, want_lse = call(q)
    ref = R.attention(host(pool), q.cpu(), rs, table, segs, None if grouped else lim,
                      groups=([0, len(rows)], ptable, [20]) if grouped else None, dtype=dtype)
    check_rows(want, ref, want_lse)
    bad = q.clone()
    marked = torch.zeros(n, hq, dtype=torch.bool, device=DEV)
    for i, (r, h) in enumerate([(0, 0), (n - 1, hq - 1), (n // 2, hq // 2)]):
        bad[r, h, i * 5] = [math.nan, math.nan, math.inf][i]
        if i == 2:
            bad[r, h, i * 5 + 1] = -math.inf         # some scores are inf - inf
        marked[r, h] = lim[r] > 0
    out, lse = call(bad)
    assert torch.isnan(out[marked]).all() and torch.isnan(lse[marked]).all()
    # (not the same bits: rows of a warp take new maxima over together)
    check_rows(torch.where(marked[..., None], want, out), ref, torch.where(marked, want_lse, lse))
    if n > 1 and not grouped:
        assert (out[n - 1] == 0).all() and (lse[n - 1] == -math.inf).all()
    assert kv.device_status() == 0
