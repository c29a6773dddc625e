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


# ------------------------------------------------------------------ keys and values that are not finite
def attention_of_marked(q, k, v, seen, hkv, dtype):
    """One sequence: q [rows][Hq][D], k and v [keys][Hkv][D] in float64 that need not be finite,
    seen [rows][keys].  Returns out, lse, their bounds as in paged_ref, and where out is not
    finite: a score of NaN or plus infinity spoils its row and head, a value its column, in the
    rows that see it; a score of minus infinity has weight zero."""
    G, D = q.shape[1] // hkv, q.shape[2]
    q = q.to(R.F64).reshape(len(q), hkv, G, D)
    x = torch.einsum("rhgd,khd->rhgk", q, k) * D ** -0.5
    x = torch.where(seen[:, None, None], x, -math.inf)
    size = torch.einsum("rhgd,khd->rhgk", q.abs(), k.abs()) * D ** -0.5
    B = torch.where(torch.isfinite(x), size, torch.zeros_like(size)).amax(3)
    lost = (torch.isnan(x) | (x == math.inf)).any(3)
    x = torch.where(lost[..., None], torch.zeros_like(x), x)
    z = torch.logsumexp(x, 3)
    w = torch.where(torch.isfinite(z)[..., None], torch.exp(x - z[..., None]), torch.zeros_like(x))
    fine = torch.isfinite(v)
    vf = torch.where(fine, v, torch.zeros_like(v))
    o, A = torch.einsum("rhgk,khd->rhgd", w, vf), torch.einsum("rhgk,khd->rhgd", w, vf.abs())
    spoilt = torch.einsum("rk,khd->rhd", seen.to(R.F64), (~fine).to(R.F64))[:, :, None] > 0
    spoilt = spoilt | lost[..., None]
    e = R.EPS[dtype]
    shift = 2 * D * 2.0 ** -23 * B + 2.0 ** -16
    sub = seen.sum(1)[:, None, None, None] * 2.0 ** -25 * vf.abs().amax() if dtype == HF else 0.0
    tol = e / 2 * o.abs() + (e / 2 + shift[..., None]) * A * (1 + e) + sub + 2.0 ** -25
    return [t.flatten(1, 2) for t in (o, z, tol, shift, spoilt, lost)]


def run_spoilt(dtype, D, hq, hkv, ps, layout, rows, segs, bad, limit=None, groups=None, seed=0):
    """bad: (sequence, position, "k" or "v", column, value): an element of one kv head of a
    sequence's own keys or values.  Only the rows that see it may change."""
    g = _gen(seed + D + sum(rows))
    top = [max(a + n for a, n in sg) for sg in segs]
    pre = groups[1] if groups else []
    n_pages = sum(-(-n // ps) for n in top + pre) + 2
    pool = make_pool(g, n_pages, hkv, ps, D, dtype, layout)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, at = make_tables(top, ps, order)
    ptable, _ = make_tables(pre, ps, order, at) if groups else (None, at)
    n = sum(rows)
    rs = [sum(rows[:i]) for i in range(len(rows) + 1)]
    q = torch.randn(n, hq, D, generator=g).to(dtype).to(DEV)
    lim = None if limit is None else [limit(s, j) for s in range(len(rows)) for j in range(rows[s])]
    for s, p, what, col, value in bad:
        pool[what == "v"][int(table[s, p // ps]), (p + col) % hkv, p % ps, col] = value
    pages, ref = host(pool), []
    for s in range(len(rows)):
        if not rows[s]:
            continue
        own = R.seq_positions(segs[s], table.shape[1] * ps)
        k, v = pages.gather(table[s], own)
        seen = torch.ones(rows[s], len(own), dtype=torch.bool)
        if lim is not None:
            seen = own[None] < torch.tensor(lim[rs[s]:rs[s + 1]])[:, None]
        if groups:
            i = [i for i in range(len(pre)) if groups[0][i] <= s < groups[0][i + 1]][0]
            pk, pv = pages.gather(ptable[i], torch.arange(pre[i]))
            k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
            seen = torch.cat([torch.ones(rows[s], pre[i], dtype=torch.bool), seen], 1)
        ref.append(attention_of_marked(q[rs[s]:rs[s + 1]].cpu(), k.transpose(0, 1), v.transpose(0, 1), seen, hkv, dtype))
    o, z, tol, ztol, spoilt, lost = (torch.cat(x) for x in zip(*ref))
    kv = make_kv(pool, hq, n, len(pre))
    out, lse = torch.full_like(q, 3.0), torch.full((n, hq), 5.0, device=DEV)
    a = (q, ints(rs), table.to(DEV), ints(segs))
    kw = dict(row_limit=None if lim is None else ints(lim), out=out, lse=lse)
    for _ in range(2):      # the second call finds what the first one left in the workspace
        if groups:
            kv.shared_prefix_attn(*a, ints(groups[0]), ptable.to(DEV), ints(pre), **kw)
        else:
            kv.attn(*a, **kw)
        got, got_lse = out.cpu().to(R.F64), lse.cpu().to(R.F64)
        assert not torch.isfinite(got[spoilt]).any()
        assert torch.isfinite(got[~spoilt]).all()
        assert ((got - o).abs() <= tol)[~spoilt].all()
        assert torch.isnan(got_lse[lost]).all()
        none = torch.isinf(z) & ~lost
        assert (got_lse[none] == -math.inf).all()
        assert ((got_lse - z).abs() <= ztol)[~lost & ~none].all()
    assert kv.device_status() == 0


NAN, INF = math.nan, math.inf


def every(s, n, D, step=1):
    """All keys and values of a sequence's first n positions, in columns that differ."""
    return [(s, p, what, (p * 5 + (what == "v")) % D, NAN if p % 3 else -INF) for p in range(0, n, step) for what in "kv"]


SPOILT = [  # dtype, D, Hq, Hkv, page, layout, rows, own segments, bad places, (first sequences, prefix lengths)
    (BF, 128, 28, 4, 16, "heads", [1, 1, 1], whole(1, 40, 300),
     [(1, 5, "v", 3, NAN), (2, 299, "v", 127, INF), (2, 0, "v", 64, -INF)], ([0, 3], [500])),
    (BF, 128, 28, 4, 16, "heads", [1, 1, 1], whole(40, 40, 300),
     [(0, 39, "k", 3, NAN), (2, 150, "k", 100, INF), (2, 151, "v", 0, NAN)], ([0, 3], [70])),
    (HF, 128, 32, 32, 64, "slots", [32, 7, 32], whole(32, 100, 64), [(1, 99, "v", 1, INF)] + every(2, 64, 128),
     ([0, 3], [130])),
    (HF, 64, 8, 2, 32, "paired", [5, 0, 70, 3, 9], whole(20, 0, 400, 33, 0),
     [(0, 19, "v", 63, NAN), (2, 399, "v", 0, INF), (2, 130, "v", 33, INF), (3, 0, "k", 0, NAN)], ([0, 5], [77])),
    (BF, 64, 4, 4, 16, "padded", [2, 2, 2], whole(200, 500, 3), every(1, 500, 64, 7), ([0, 3], [1])),
    (HF, 32, 4, 4, 8, "padded", [8, 8, 8, 8], whole(8, 60, 8, 130), [(3, 129, "v", 31, NAN), (1, 7, "v", 0, -INF)],
     ([0, 4], [257])),
    (BF, 32, 6, 1, 8, "heads", [40, 30], whole(140, 60), every(0, 140, 32, 9), ([0, 2], [30])),
    # own lists that are cut over many CTAs
    (BF, 128, 7, 1, 128, "heads", [1, 1, 1], whole(9000, 300, 1),
     [(0, 8999, "v", 7, NAN), (0, 4000, "v", 8, INF), (0, 3000, "v", 8, -INF)], ([0, 3], [1000])),
    (HF, 64, 14, 2, 64, "slots", [20, 9], whole(300, 20000), [(1, p, "v", p % 64, INF) for p in range(0, 20000, 997)],
     ([0, 2], [400])),
]


@pytest.mark.parametrize("case", SPOILT, ids=lambda c: str(c)[:60])
def test_sequences_of_a_group_do_not_spoil_each_other(case):
    run_spoilt(*case[:9], groups=case[9])


@pytest.mark.parametrize("case", [
    (BF, 128, 28, 4, 16, "heads", [1, 3, 4], whole(300, 129, 128)),         # 32-row tiles
    (HF, 64, 8, 2, 64, "slots", [70, 133], whole(700, 390)),                # 128-row tiles
    (BF, 32, 4, 4, 8, "padded", [30, 17], whole(300, 40)),
    (HF, 128, 4, 1, 32, "paired", [33], [((200, 300), (10, 50))]),
    (BF, 128, 4, 4, 64, "heads", [200, 70], whole(400, 5000)),
], ids=lambda c: str(c)[:60])
@pytest.mark.parametrize("grouped", [False, True])
def test_later_keys_do_not_spoil_earlier_rows(case, grouped):
    """Under a causal limit a row is the same whatever the positions beyond its own hold."""
    rows, end = case[6], [max(a + n for a, n in sg) for sg in case[7]]
    D, bad = case[1], []
    for s, m in enumerate(rows):
        bad += [(s, end[s] - 1 - j, "kv"[(j + 1) % 2], (11 * j + s) % D, [NAN, INF, -INF][j % 3])
                for j in range(0, m, max(1, m // 4)) if any(a <= end[s] - 1 - j < a + n for a, n in case[7][s])]
    run_spoilt(*case, bad, limit=lambda s, j: end[s] - rows[s] + j + 1,
               groups=([0, len(rows)], [150]) if grouped else None)


@pytest.mark.parametrize("case", [
    # a key of score minus infinity for some heads, alone in its part of a cut tile; its value counts in whole and
    # in cut tiles alike
    (BF, 64, 16, 8, 256, "heads", [2], whole(1), [(0, 0, "k", 53, INF), (0, 0, "v", 45, NAN)], ([0, 1], [1])),
    (HF, 64, 8, 1, 1024, "heads", [1, 33], whole(300, 1), [(1, 0, "k", 46, -INF), (1, 0, "v", 56, -INF)], ([0, 2], [1])),
    (HF, 128, 8, 8, 256, "padded", [1, 2], [((0, 129), (0, 0)), ((187, 1), (233, 1))],
     [(1, 187, "k", 99, INF), (1, 187, "v", 27, NAN), (1, 187, "v", 107, INF)], None),
    (BF, 128, 4, 1, 64, "slots", [1], whole(20000), [(0, p, w, 7, INF) for p in range(0, 20000, 64) for w in "kv"], None),
], ids=lambda c: str(c)[:60])
def test_values_of_keys_that_weigh_nothing_count(case):
    run_spoilt(*case[:9], groups=case[9])


# ------------------------------------------------------------------ waits that run out
def c_call(pool, q, out, rs, table):
    """Argument blocks of the C calls over these tensors."""
    import ctypes as C

    from diffusion_decoding_step_b200 import abi
    k, v = pool
    kv = abi.dllm_kv_pages(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), k.shape[0], k.shape[2],
                           k.shape[1], k.shape[3], int(k.dtype is HF))
    bt = abi.dllm_paged_batch(len(rs) - 1, q.shape[0], table.shape[1], table.stride(0), rs.data_ptr(), table.data_ptr())
    rows = [abi.dllm_rows(x.data_ptr(), x.stride(0), x.stride(1)) for x in (q, out)]
    return [C.byref(x) for x in (kv, bt, *rows)]


@pytest.mark.parametrize("where", [0, 1, 2])
@pytest.mark.parametrize("case", [
    (BF, 128, 28, 4, 16, [1], [40000]),         # 32-row tiles, cut over all CTAs
    (HF, 64, 8, 2, 64, [70, 133], [700, 390]),  # 128-row tiles
    (BF, 32, 4, 1, 8, [1], [5]),                # one working CTA
], ids=lambda c: str(c)[:60])
def test_waits_that_run_out_are_reported(case, where):
    """Something is held back in each working block, with a limit of 20 ms: the call reports it
    and returns, and the next calls, this kernel's on the same workspace among them, are right."""
    import ctypes as C
    import time

    from diffusion_decoding_step_b200 import abi
    from tests.gpu_util import ptr, stream
    dtype, D, hq, hkv, ps, rows, lens = case
    g = _gen(5)
    n_pages = sum(-(-n // ps) for n in lens) + 1
    pool = make_pool(g, n_pages, hkv, ps, D, dtype, "heads")
    table, _ = make_tables(lens, ps, torch.randperm(n_pages, generator=g).to(torch.int32))
    n, rs = sum(rows), [sum(rows[:i]) for i in range(len(rows) + 1)]
    q = torch.randn(n, hq, D, generator=g).to(dtype).to(DEV)
    out, segs, r, t = torch.zeros_like(q), ints(whole(*lens)), ints(rs), table.to(DEV)
    kv = make_kv(pool, hq, n)
    want = kv.attn(q, r, t, segs)
    a, b, qr, orow = c_call(pool, q, out, r, t)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    abi.check(abi.dllm_selftest_paged_timeout(a, b, hq, ptr(segs), qr, orow, ptr(kv.ws), kv.ws.numel(), where, 20000,
                                              stream()), "selftest")
    torch.cuda.synchronize()
    assert 0.015 <= time.perf_counter() - t0 < 5.0
    assert kv.device_status() == abi.DLLM_DEVICE_TIMEOUT
    abi.check(abi.dllm_paged_workspace_init(ptr(kv.ws), kv.ws.numel(), stream()), "init")
    assert torch.equal(kv.attn(q, r, t, segs), want)
    assert kv.device_status() == 0
    check_rows(want, R.attention(host(pool), q.cpu(), rs, table, whole(*lens), dtype=dtype))


def test_the_timeout_selftest_checks_its_arguments():
    from diffusion_decoding_step_b200 import abi
    from tests.gpu_util import ptr, stream
    g = _gen(6)
    pool = make_pool(g, 2, 1, 16, 64, BF, "heads")
    kv = make_kv(pool, 1, 1)
    q = torch.zeros(1, 1, 64, dtype=BF, device=DEV)
    out, r, t, segs = torch.zeros_like(q), ints([0, 1]), ints([[0]]), ints(whole(3))
    a, b, qr, orow = c_call(pool, q, out, r, t)
    for where, limit in ((-1, 20), (3, 20), (0, 0), (0, 1000001)):
        assert abi.dllm_selftest_paged_timeout(a, b, 1, ptr(segs), qr, orow, ptr(kv.ws), kv.ws.numel(), where, limit,
                                               stream()) == abi.DLLM_ERR_INVALID
    assert abi.dllm_selftest_paged_timeout(None, b, 1, ptr(segs), qr, orow, ptr(kv.ws), kv.ws.numel(), 0, 20,
                                           stream()) == abi.DLLM_ERR_INVALID
    assert kv.device_status() == 0


# ------------------------------------------------------------------ what PagedKV takes
def small(groups=None, **kw):
    """A PagedKV over four pages and the arguments of an attention call of three rows."""
    from diffusion_decoding_step_b200.paged import PagedKV
    g = _gen(24)
    pool = make_pool(g, 4, 2, 16, 64, BF, "heads")
    kv = PagedKV(pool[0], pool[1], 4, 3) if groups is None else PagedKV(pool[0], pool[1], 4, 3, groups)
    q = torch.randn(3, 4, 64, generator=g).to(BF).to(DEV)
    return pool, kv, q, (ints([0, 1, 3]), ints([[0, 1], [2, 0]]), ints(whole(20, 7)))


def test_prefix_groups_need_no_announcement():
    pool, kv, q, a = small()
    pt, n = torch.tensor([[3], [1]], dtype=torch.int32), [9, 16]
    out = kv.shared_prefix_attn(q, *a, ints([0, 1, 2]), pt.to(DEV), ints(n))
    check_rows(out, R.attention(host(pool), q.cpu(), [0, 1, 3], a[1].cpu(), whole(20, 7), groups=([0, 1, 2], pt, n)))
    assert kv.device_status() == 0


def test_announced_prefix_groups_are_the_most():
    _, kv, q, a = small(1)
    g2 = (ints([0, 1, 2]), ints([[3], [1]]), ints([9, 16]))
    with pytest.raises(ValueError, match="2 prefix groups.* 1"):
        kv.shared_prefix_attn(q, *a, *g2)
    _, kv, q, a = small(0)
    with pytest.raises(ValueError, match="without prefix groups"):
        kv.shared_prefix_attn(q, *a, *g2)
    with pytest.raises(ValueError, match="without prefix groups"):
        kv.shared_prefix_attn(q, *a, ints([0]), g2[1][:0], g2[2][:0])
    _, kv, q, a = small()
    with pytest.raises(ValueError, match="group_start"):
        kv.shared_prefix_attn(q, *a, ints([0]), g2[1][:0], g2[2][:0])


def test_a_call_without_rows_does_nothing():
    pool, kv, q, a = small()
    start = [x.clone() for x in pool]
    k = torch.zeros(0, 2, 64, dtype=BF, device=DEV)
    rs, rs0 = ints([0, 0, 0]), ints([0])
    launched = None
    from diffusion_decoding_step_b200 import abi
    torch.cuda.synchronize()
    launched = abi.dllm_launch_count()
    for r, tab, segs, pos in ((rs, a[1], a[2], ints([5, 3])), (rs0, a[1][:0], a[2][:0], ints([]))):
        assert kv.attn(q[:0], r, tab, segs).shape == (0, 4, 64)
        assert kv.attn(q[:0], r, tab, segs, row_limit=ints([]), out=q[:0], lse=torch.zeros(0, 4, device=DEV)) is not None
        assert kv.shared_prefix_attn(q[:0], r, tab, segs, ints([0, 0]), ints([[3]]), ints([9])).shape == (0, 4, 64)
        assert kv.append(k, k, r, tab, pos, q=q[:0], rope_theta=1e4).shape == (0, 4, 64)
        assert kv.append(k, k, r, tab, pos) is None
    assert abi.dllm_launch_count() == launched
    assert all(torch.equal(x, y) for x, y in zip(pool, start)) and kv.device_status() == 0
    # the arguments are checked all the same
    for f in (lambda: kv.attn(q[:0], rs, a[1], a[2][:1]), lambda: kv.append(k, k.half(), rs, a[1], ints([0, 0])),
              lambda: kv.attn(q[:0], rs, a[1], a[2], row_limit=ints([1]))):
        with pytest.raises(ValueError):
            f()


def test_numbers_that_do_not_fit_are_refused():
    """Not cut to 32 bits, nor rounded to the zero that stands for the default."""
    from diffusion_decoding_step_b200.paged import PagedKV
    pool, kv, q, a = small()
    for f in (lambda: PagedKV(*pool, 2 ** 32 + 4, 3), lambda: PagedKV(*pool, 4, 2 ** 32 + 3),
              lambda: PagedKV(*pool, 4, 3, 2 ** 32 + 1), lambda: PagedKV(*pool, 4, 3, -1),
              lambda: PagedKV(*pool, 4, 2 ** 31)):
        with pytest.raises(ValueError, match="n_q_heads|max_rows|max_groups"):
            f()
    k, pos = torch.zeros(3, 2, 64, dtype=BF, device=DEV), ints([0, 0])
    for tiny in (1e-46, 1e-300):
        with pytest.raises(ValueError, match="scale"):
            kv.attn(q, *a, scale=tiny)
        with pytest.raises(ValueError, match="scale"):
            kv.shared_prefix_attn(q, *a, ints([0, 2]), ints([[3]]), ints([9]), scale=tiny)
        with pytest.raises(ValueError, match="rope_theta"):
            kv.append(k, k, a[0], a[1], pos, rope_theta=tiny)
    kv.attn(q, *a, scale=1e-40)
    assert kv.device_status() == 0


def test_no_gradients_are_dropped_in_silence():
    pool, kv, q, a = small()
    k, pos, out = torch.ones(3, 2, 64, dtype=BF, device=DEV), ints([0, 3]), torch.zeros_like(q)
    qg, kg = q.clone().requires_grad_(), k.clone().requires_grad_()
    calls = [lambda: kv.attn(qg, *a), lambda: kv.attn(q, *a, out=qg.clone()),
             lambda: kv.shared_prefix_attn(qg, *a, ints([0, 2]), ints([[3]]), ints([9])),
             lambda: kv.append(kg, k, a[0], a[1], pos), lambda: kv.append(k, kg * 2, a[0], a[1], pos),
             lambda: kv.append(k, k, a[0], a[1], pos, q=qg, q_out=out)]
    for f in calls:
        with pytest.raises(ValueError, match="no backward"):
            f()
        with torch.no_grad():
            f()
    with torch.inference_mode():
        kv.attn(qg, *a)
    from diffusion_decoding_step_b200.paged import PagedKV
    with pytest.raises(ValueError, match="gradient"):
        PagedKV(pool[0].clone().requires_grad_(), pool[1].clone().requires_grad_(), 4, 3)


def test_autograd_sees_what_a_call_has_written():
    """Tensors that a backward pass has saved and that a call overwrites are refused there."""
    pool, kv, q, a = small()
    k, pos = torch.ones(3, 2, 64, dtype=BF, device=DEV), ints([0, 3])
    out, lse, q_out = torch.ones_like(q), torch.ones(3, 4, device=DEV), torch.ones_like(q)
    writes = [(pool[0], lambda: kv.append(k, k, a[0], a[1], pos)), (pool[1], lambda: kv.append(k, k, a[0], a[1], pos)),
              (q_out, lambda: kv.append(k, k, a[0], a[1], pos, q=q, q_out=q_out)),
              (out, lambda: kv.attn(q, *a, out=out, lse=lse)), (lse, lambda: kv.attn(q, *a, out=out, lse=lse))]
    for x, f in writes:
        w = torch.ones_like(x, requires_grad=True)
        y = (x * w).float().sum()
        f()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    y = (q * torch.ones_like(q, requires_grad=True)).float().sum()
    kv.attn(q, *a)
    y.backward()            # what is only read is as it was
    y = (pool[0] * torch.ones_like(pool[0], requires_grad=True)).float().sum()
    kv.append(k[:0], k[:0], ints([0, 0, 0]), a[1], pos)
    y.backward()            # and so is everything after a call without rows
    with torch.inference_mode():
        o = torch.zeros_like(q)
        kv.attn(q, *a, out=o)       # tensors without a version counter


# ------------------------------------------------------------------ bounds
class Guarded:
    """Tensors inside one buffer of a byte pattern, 64 KiB and more between them."""
    GAP, PATTERN = 65536, 0xA5

    def __init__(self, total):
        self.buf = torch.full((total,), self.PATTERN, dtype=torch.uint8, device=DEV)
        self.at, self.parts = self.GAP, []

    def put(self, x):
        n = x.numel() * x.element_size()
        view = self.buf[self.at:self.at + n].view(x.dtype).view(x.shape)
        view.copy_(x)
        self.parts.append((self.at, self.at + n))
        self.at = (self.at + n + self.GAP + 1023) // 1024 * 1024
        assert self.at <= self.buf.numel()
        return view

    def check(self):
        edge = 0
        for a, b in self.parts + [(self.buf.numel(), 0)]:
            assert bool((self.buf[edge:a] == self.PATTERN).all()), f"written between bytes {edge} and {a}"
            edge = b


def steps_up(v, hi):
    """What the kernels make of starts that may hold anything: clamped, then non-decreasing."""
    out = []
    for x in v:
        out.append(max([min(max(x, 0), hi)] + out[-1:]))
    return out


WILD = [[-5, 3, 100], [8, 4, 0], [2 ** 31 - 1, LOW, 2 ** 31 - 1], [0, 8, 8], [5, 5, 6], [LOW, LOW, 7], [3, 0, 6]]


@pytest.mark.parametrize("hq,hkv,D,dtype", [(2, 1, 64, BF), (28, 4, 128, HF), (6, 6, 32, BF)])
def test_attention_with_any_starts_writes_only_its_outputs(hq, hkv, D, dtype):
    """Any contents of row_start and group_start: nothing but out, lse and the workspace changes,
    and the rows are those of the starts made non-decreasing."""
    import ctypes as C

    from diffusion_decoding_step_b200 import abi
    from tests.gpu_util import ptr, stream
    g = _gen(11)
    n = 8
    pool = make_pool(g, 12, hkv, 16, D, dtype, "heads")
    table, ptab = torch.tensor([[0, 1, 9], [2, 3, 10]], dtype=torch.int32), torch.tensor([[4], [5]], dtype=torch.int32)
    segs, plen = whole(40, 32), [9, -4]
    gd = Guarded(64 << 20)
    k, v = gd.put(pool[0]), gd.put(pool[1])
    kept = [k.clone(), v.clone()]
    q = gd.put(torch.randn(n, hq, D, generator=g).to(dtype).to(DEV))
    out, lse = gd.put(torch.full_like(q, 7.0)), gd.put(torch.full((n, hq), 5.0, device=DEV))
    t, pt, sg, pl = (gd.put(x.to(DEV)) for x in (table, ptab, ints(segs), ints(plen)))
    rs, gs = gd.put(ints([0] * 3)), gd.put(ints([0] * 3))
    a, b, qr, orow = c_call((k, v), q, out, rs, t)
    size = C.c_size_t(0)
    abi.check(abi.dllm_paged_workspace_size(a, hq, n, C.byref(size)), "size")
    ws = gd.put(torch.zeros(size.value, dtype=torch.uint8, device=DEV))
    grp = abi.dllm_prefix_groups(2, 1, pt.stride(0), gs.data_ptr(), pt.data_ptr(), pl.data_ptr())
    abi.check(abi.dllm_paged_workspace_init(ptr(ws), size.value, stream()), "init")
    pages = R.Pages(*[x.cpu().to(R.F64) for x in kept])

    def one(starts, groups):
        out.fill_(7.0), lse.fill_(5.0), rs.copy_(ints(starts))
        if groups is None:
            abi.check(abi.dllm_paged_attn(a, b, hq, ptr(sg), None, 0.0, qr, orow, ptr(lse), ptr(ws), size.value,
                                          stream()), "attn")
        else:
            gs.copy_(ints(groups))
            abi.check(abi.dllm_shared_prefix_attn(a, b, C.byref(grp), hq, ptr(sg), None, 0.0, qr, orow, ptr(lse),
                                                  ptr(ws), size.value, stream()), "shared")
        up = steps_up(starts, n)
        ref = R.attention(pages, q.cpu(), up, table, segs, dtype=dtype,
                          groups=None if groups is None else (steps_up(groups, 2), ptab, plen))
        check_rows(out, ref, lse, torch.full_like(out, 7.0))
        gd.check()
        assert torch.equal(k, kept[0]) and torch.equal(v, kept[1])

    for starts in WILD:
        one(starts, None)
        for groups in ([0, 1, 2], [-4, 7, 1], [2 ** 31 - 1, LOW, 5], [1, 0, 2]):
            one(starts, groups)
    code = C.c_int32(0)
    abi.check(abi.dllm_device_status(ptr(ws), C.byref(code), stream()), "status")
    assert code.value == 0


@pytest.mark.parametrize("hq,hkv,D,dtype", [(2, 1, 64, BF), (28, 4, 128, HF)])
def test_append_with_any_starts_writes_only_its_outputs(hq, hkv, D, dtype):
    """Any contents of row_start, pos and the table: nothing outside the pages and q_out changes,
    and the pages only in slots that a table row reaches."""
    import ctypes as C

    from diffusion_decoding_step_b200 import abi
    from tests.gpu_util import ptr, stream
    g = _gen(12)
    n = 8
    gd = Guarded(32 << 20)
    pool = [gd.put(x) for x in make_pool(g, 6, hkv, 16, D, dtype, "heads")]
    rows = [gd.put(torch.randn(n, h, D, generator=g).to(dtype).to(DEV)) for h in (hq, hkv, hkv)]
    q_out = gd.put(torch.zeros(n, hq, D, dtype=dtype, device=DEV))
    kept = [x.clone() for x in pool]
    rs, pos, t = gd.put(ints([0] * 3)), gd.put(ints([0] * 2)), gd.put(ints([[0, 1], [2, 3]]))
    status = gd.put(ints([0]))
    a, b, q, o = c_call(pool, rows[0], q_out, rs, t)
    k, v = (C.byref(abi.dllm_rows(x.data_ptr(), x.stride(0), x.stride(1))) for x in rows[1:])
    for table in ([[0, 1], [2, 3]], [[-1, 6], [2 ** 31 - 1, LOW]], [[0, 99], [-7, 3]]):
        for starts in WILD:
            for where in ([0, 0], [15, 30], [LOW, 2 ** 31 - 1], [-3, 29]):
                rs.copy_(ints(starts)), pos.copy_(ints(where)), t.copy_(ints(table))
                abi.check(abi.dllm_paged_append(a, b, hq, q, k, v, o, ptr(pos), None, 1e4, ptr(status), stream()),
                          "append")
    gd.check()
    for x, y in zip(pool, kept):
        assert torch.equal(x[4:], y[4:])        # pages that no table row names


def test_workspaces_and_tables_may_be_larger():
    for c in (SHARED[0], SHARED[1], SHARED[8]):
        run_attn(*c[:8], groups=c[8], kv_rows=5000, width=40)
        run_attn(*c[:8], kv_rows=700, width=25)


# ------------------------------------------------------------------ as they are used
def test_growth_over_steps_matches_the_contiguous_cache():
    """Two prompts of different lengths enter, then each sequence grows by three blocks: after
    every append the attention gives what dllm_block_attn gives over the same keys."""
    import ctypes as C

    from diffusion_decoding_step_b200 import abi
    from diffusion_decoding_step_b200 import workload as wl
    from diffusion_decoding_step_b200.runtime import make_config, workspace_bytes
    from tests.gpu_util import ptr, stream
    g = _gen(41)
    hq, hkv, D, ps, B, steps, prompts = 28, 4, 128, 16, 32, 3, [200, 57]
    ends = [p + steps * B for p in prompts]
    pool = make_pool(g, 60, hkv, ps, D, BF, "slots")
    table, _ = make_tables(ends, ps, torch.randperm(60, generator=g).to(torch.int32))
    tab = table.to(DEV)
    kv = make_kv(pool, hq, sum(prompts))
    w = wl.Workload("t", batch=2, n_layers=1, hidden=512, n_q_heads=hq, n_kv_heads=hkv, head_dim=D, vocab=1024,
                    prompt_len=224, gen_len=steps * B, block=B)
    cfg, size = make_config(w), workspace_bytes(w)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    abi.check(abi.dllm_workspace_init(C.byref(cfg), ptr(ws), size, stream()), "ws init")
    kc = torch.zeros(1, 2, hkv, w.seq_len, D, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)

    def rows(n):
        x = torch.randn(n, hq + 2 * hkv, D, generator=g).to(BF).to(DEV)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    _, k, v = rows(sum(prompts))
    kv.append(k, v, ints([0, prompts[0], sum(prompts)]), tab, ints([0, 0]), rope_theta=1e6)
    rs = [0, B, 2 * B]
    for step in range(steps):
        at = [p + step * B for p in prompts]
        lens = [n + B for n in at]
        q, k, v = rows(2 * B)
        q = kv.append(k, v, ints(rs), tab, ints(at), q=q, rope_theta=1e6)
        out = kv.attn(q, ints(rs), tab, ints(whole(*lens)))
        pages = host(pool)
        for s in range(2):      # the same keys in the contiguous cache
            for cache, x in zip((kc, vc), pages.gather(table[s], torch.arange(lens[s]))):
                cache[0, s, :, :lens[s]] = x.to(BF).to(DEV)
        qb = q.reshape(2, B, hq, D).transpose(1, 2).contiguous()
        want = torch.empty(2 * B, hq * D, dtype=BF, device=DEV)
        abi.check(abi.dllm_block_attn(C.byref(cfg), 0, B, ptr(qb), ptr(kc), ptr(vc), ptr(ints(whole(*lens))), ptr(want),
                                      ptr(ws), size, stream()), "attn")
        torch.cuda.synchronize()
        ref = R.attention(pages, q.cpu(), rs, table, whole(*lens))
        check_rows(out, ref)
        check_rows(want.reshape(2 * B, hq, D), ref)
    assert kv.device_status() == 0
