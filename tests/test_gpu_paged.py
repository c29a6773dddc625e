"""The paged cache operators against their 64-bit definitions (B200 only)."""
import math
import random

import pytest
import torch

from tests import paged_ref as R
from tests.gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def make_pool(g, n, hkv, ps, D, dtype, layout):
    """k, v views [n][hkv][ps][D] on the GPU in one of several memory orders."""
    ensure_lib()
    vals = [torch.randn(n, hkv, ps, D, generator=g).to(dtype).to(DEV) for _ in range(2)]
    if layout == "heads":
        return vals
    if layout == "slots":
        return [x.transpose(1, 2).contiguous().transpose(1, 2) for x in vals]
    if layout == "paired":       # keys and values of a page side by side
        both = torch.stack(vals, 1)
        return [both[:, 0], both[:, 1]]
    if layout == "padded":       # rows of D + 8 elements, heads of ps + 1 slots
        out = []
        for x in vals:
            big = torch.full((n, hkv, ps + 1, D + 8), float("nan"), dtype=dtype, device=DEV)
            big[:, :, :ps, :D] = x
            out.append(big[:, :, :ps, :D])
        return out
    raise ValueError(layout)


def make_kv(pool, hq, rows, groups=0):
    from diffusion_decoding_step_b200.paged import PagedKV
    return PagedKV(pool[0], pool[1], hq, rows, groups)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def host(pool):
    return R.Pages(*[x.cpu().to(R.F64) for x in pool])


def make_tables(lens, ps, order, at=0, width=None):
    """Page lists of the lengths (and -1 behind), taking pages from order[at:]."""
    counts = [-(-n // ps) for n in lens]
    width = width or max(counts + [1])
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    for i, c in enumerate(counts):
        t[i, :c] = order[at:at + c]
        at += c
    return t, at


def check_rows(out, ref, lse=None, untouched=None):
    o = out.cpu().to(R.F64)
    for r, (want, z, tol, ztol) in ref.items():
        err = (o[r] - want).abs()
        assert not torch.isnan(o[r]).any(), f"row {r}: NaN"
        assert (err <= tol).all(), \
            f"row {r}: off by {err.max():.3g}, {float((err / tol).max()):.2f} of what is allowed"
        if lse is not None:
            got = lse[r].cpu().to(R.F64)
            fin = torch.isfinite(z)
            assert torch.equal(torch.isfinite(got), fin) and (got[~fin] == -math.inf).all()
            assert ((got - z).abs()[fin] <= ztol[fin]).all(), f"row {r}: lse"
    if untouched is not None:
        for r in range(o.shape[0]):
            if r not in ref:
                assert torch.equal(out[r].cpu(), untouched[r].cpu()), f"row {r} was written"


# ------------------------------------------------------------------ append
APPEND = [  # dtype, D, Hq, Hkv, page, layout, rows per sequence, first positions, shifts
    (BF, 128, 28, 4, 16, "heads", [1], [0], None),
    (BF, 128, 32, 32, 64, "slots", [32, 0, 5, 31], [100, 7, 63, 1], [0, 0, -3, 12]),
    (HF, 128, 7, 1, 8, "paired", [1, 1, 1, 1, 1], [0, 7, 8, 9, 100], [5, -100, 0, 1, 2]),
    (HF, 64, 8, 2, 128, "heads", [130, 3], [1, 255], None),
    (BF, 32, 4, 4, 32, "padded", [9, 64, 0], [0, 31, 5], [1, 2, 3]),
    (BF, 64, 1, 1, 1024, "slots", [1, 40], [1023, 1000], None),
    (HF, 32, 16, 1, 256, "padded", [17], [250], [1000000]),
]


def run_append(dtype, D, hq, hkv, ps, layout, rows, pos, shift, theta=1e6, q_mode="packed", seed=0,
               before=2, behind=3):
    g = _gen(seed + D + ps)
    ends = [p + n for p, n in zip(pos, rows)]
    n_pages = sum(-(-max(e, 1) // ps) for e in ends) + 2
    pool = make_pool(g, n_pages, hkv, ps, D, dtype, layout)
    start = host(pool)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, _ = make_tables([max(e, 1) for e in ends], ps, order)
    n = before + sum(rows) + behind
    row_start = [before + sum(rows[:i]) for i in range(len(rows) + 1)]
    packed = torch.randn(n, hq + 2 * hkv, D, generator=g).to(dtype).to(DEV)
    packed[row_start[-1]:] = float("nan")       # rows of no sequence are not looked at
    packed[:before] = float("nan")
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    x = [t.cpu().to(R.F64) for t in (q, k, v)]
    kv = make_kv(pool, hq, n)
    if q_mode == "packed":
        out = torch.full((n, hq, D), 7.0, dtype=dtype, device=DEV)
        got = kv.append(k, v, ints(row_start), table.to(DEV), ints(pos), q=q, q_out=out,
                        rope_theta=theta, rope_shift=None if shift is None else ints(shift))
    elif q_mode == "in place":
        got = kv.append(k, v, ints(row_start), table.to(DEV), ints(pos), q=q, q_out=q,
                        rope_theta=theta, rope_shift=None if shift is None else ints(shift))
    else:
        got = kv.append(k, v, ints(row_start), table.to(DEV), ints(pos), rope_theta=theta,
                        rope_shift=None if shift is None else ints(shift))
        assert got is None
    torch.cuda.synchronize()
    assert kv.device_status() == 0
    after = host(pool)
    named = torch.zeros(start.k.shape[0], ps, dtype=torch.bool)
    for s in range(len(rows)):
        for j in range(rows[s]):
            r, p = row_start[s] + j, pos[s] + j
            t = torch.tensor([p + (shift[s] if shift else 0)])
            pg, sl = int(table[s, p // ps]), p % ps
            named[pg, sl] = True
            want = R.rotate(x[1][r:r + 1], t, theta)
            err = (after.k[pg, :, sl] - want[0]).abs()
            assert (err <= R.rotate_bound(want, x[1][r:r + 1], dtype)[0]).all(), (s, j)
            assert torch.equal(after.v[pg, :, sl], x[2][r])
            if got is not None:
                want = R.rotate(x[0][r:r + 1], t, theta)
                err = (got[r].cpu().to(R.F64) - want[0]).abs()
                assert (err <= R.rotate_bound(want, x[0][r:r + 1], dtype)[0]).all(), (s, j)
    keep = ~named[:, None, :, None].expand_as(start.k)
    assert torch.equal(after.k[keep], start.k[keep]) and torch.equal(after.v[keep], start.v[keep])
    if q_mode == "packed":
        lost = [r for r in range(n) if r < row_start[0] or r >= row_start[-1]]
        assert (got[lost] == 7.0).all()
    elif q_mode == "in place":
        assert torch.equal(packed[:, hq:].nan_to_num(nan=9.0).cpu().to(R.F64),
                           torch.cat(x[1:], 1).nan_to_num(nan=9.0))


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(case):
    run_append(*case)


@pytest.mark.parametrize("q_mode", ["in place", "none"])
def test_append_query_forms(q_mode):
    run_append(*APPEND[1], q_mode=q_mode)


def test_append_without_rotation_copies():
    run_append(*APPEND[1], theta=0.0)


def test_append_far_positions():
    """Angles near position 2^30 keep their fraction of a turn (64-bit reduction)."""
    run_append(BF, 128, 4, 2, 64, "heads", [3, 2], [5, 70], [2 ** 30, -(2 ** 30) - 7], theta=1e4)


def test_append_many_sequences():
    n = 700
    run_append(HF, 32, 2, 1, 8, "heads", [i % 3 for i in range(n)], [i % 11 for i in range(n)], None)


def test_append_bad_pages_and_positions():
    """Entries that name no page and positions outside the table are skipped and reported."""
    g = _gen(3)
    pool = make_pool(g, 6, 2, 16, 64, BF, "heads")
    start = [x.clone() for x in pool]
    kv = make_kv(pool, 4, 8)
    x = torch.randn(8, 8, 64, generator=g).to(BF).to(DEV)
    table = ints([[0, -1], [6, 2 ** 31 - 1], [1, 2], [3, 4]])
    pos = ints([16, 3, -1, 2 ** 31 - 1])
    q = kv.append(x[:, 4:6], x[:, 6:], ints([0, 2, 4, 6, 8]), table, pos, q=x[:, :4], rope_theta=1e4)
    assert kv.device_status() == 4
    kv2 = make_kv(pool, 4, 8)
    assert kv2.device_status() == 0
    # only position 0 (row 5) named a page of the pool
    want = start[0].clone()
    want[1, :, 0] = pool[0][1, :, 0]
    assert torch.equal(pool[0], want) and not torch.equal(pool[0], start[0])
    assert torch.equal(pool[1][1, :, 0], x[5, 6:])
    assert not torch.isnan(q).any()


def test_append_any_row_start_stays_in_bounds():
    g = _gen(4)
    pool = make_pool(g, 4, 1, 16, 32, BF, "heads")
    kv = make_kv(pool, 1, 8)
    x = torch.randn(8, 3, 32, generator=g).to(BF).to(DEV)
    for rs in ([-5, 3, 100], [8, 4, 0], [2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 1]):
        kv.append(x[:, 1:2], x[:, 2:], ints(rs), ints([[0, 1], [2, 3]]), ints([0, 0]), q=x[:, :1])
    torch.cuda.synchronize()


# ------------------------------------------------------------------ attention
def run_attn(dtype, D, hq, hkv, ps, layout, rows, segs, limit=None, groups=None, scale=0.0, seed=0,
             before=1, behind=2, nan=True, width=None, kv_rows=None, spread=1.0, caps=None, seen_only=False):
    """groups: (first sequences, prefix lengths).  seen_only: slots beyond the limits of all rows
    hold anything too."""
    g = _gen(seed + 13 * D + ps + sum(rows))
    top = [max([0] + [a + n for a, n in sg if n > 0]) for sg in segs]
    pre = groups[1] if groups else []
    n_pages = sum(-(-n // ps) for n in top + pre) + 2
    pool = make_pool(g, n_pages, hkv, ps, D, dtype, layout)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table, at = make_tables(top, ps, order, width=width)
    ptable = None
    if groups:
        ptable, at = make_tables(pre, ps, order, at)
    if nan:  # slots that no segment reaches hold anything
        used = torch.zeros(n_pages, ps, dtype=torch.bool)
        for s, sg in enumerate(segs):
            p = R.seq_positions(sg, table.shape[1] * ps)
            if seen_only:
                p = p[p < max([0] + [limit(s, j) for j in range(rows[s])])]
            used[table[s][p // ps].long(), p % ps] = True
        for i, n in enumerate(pre):
            p = torch.arange(n)
            used[ptable[i][p // ps].long(), p % ps] = True
        for j, x in enumerate(pool):
            junk = torch.tensor([math.nan, math.inf, -math.inf])[torch.randint(0, 3, used.shape, generator=g)]
            x.copy_(torch.where(used.to(DEV)[:, None, :, None], x, junk.to(dtype).to(DEV)[:, None, :, None]))
    n = before + sum(rows) + behind
    row_start = [before + sum(rows[:i]) for i in range(len(rows) + 1)]
    q = (torch.randn(n, hq + 1, D, generator=g) * spread).to(dtype).to(DEV)[:, 1:]
    q[:before] = math.nan
    q[row_start[-1]:] = math.nan
    lim = None
    if limit is not None:
        lim = [0] * before + [limit(s, j) for s in range(len(rows)) for j in range(rows[s])] + [0] * behind
    kv = make_kv(pool, hq, kv_rows or n, len(pre))
    out = torch.full((n, hq, D), 7.0, dtype=dtype, device=DEV)
    keep = out.clone()
    lse = torch.full((n, hq), 5.0, device=DEV)
    a = (q, ints(row_start), table.to(DEV), ints(segs))
    kw = dict(row_limit=None if lim is None else ints(lim), scale=scale, out=out, lse=lse)
    if groups:
        kv.shared_prefix_attn(*a, ints(groups[0]), ptable.to(DEV), ints(pre), **kw)
    else:
        kv.attn(*a, **kw)
    torch.cuda.synchronize()
    assert kv.device_status() == 0
    ref = R.attention(host(pool), q.cpu(), row_start, table, segs, lim, scale,
                      (groups[0], ptable, pre) if groups else None, dtype)
    check_rows(out, ref, lse, keep)
    for r in range(n):
        if r not in ref:
            assert (lse[r] == 5.0).all()
    first = out.clone()
    if groups:
        kv.shared_prefix_attn(*a, ints(groups[0]), ptable.to(DEV), ints(pre), **kw)
    else:
        kv.attn(*a, **kw)
    assert torch.equal(first, out)  # the same call gives the same bits


def whole(*lens):
    return [((0, n), (0, 0)) for n in lens]


ATTN = [  # dtype, D, Hq, Hkv, page, layout, rows, segments
    (BF, 128, 28, 4, 16, "heads", [1], whole(1)),
    (BF, 128, 28, 4, 16, "slots", [1, 1, 1], whole(127, 128, 129)),
    (HF, 128, 7, 1, 64, "heads", [1, 0, 2, 1], whole(0, 50, 700, 5)),
    (BF, 128, 32, 32, 64, "paired", [32, 32], whole(300, 64)),
    (HF, 128, 32, 32, 8, "heads", [5, 1], whole(33, 1000)),
    (BF, 128, 8, 8, 128, "padded", [130, 3, 128], whole(257, 511, 128)),
    (BF, 64, 8, 2, 32, "slots", [33, 70], whole(512, 100)),
    (HF, 64, 71, 1, 256, "heads", [3, 1], whole(600, 257)),
    (BF, 64, 128, 1, 1024, "padded", [2, 1], whole(1500, 1)),
    (BF, 32, 4, 4, 16, "heads", [8, 64, 1], whole(72, 200, 9)),
    (HF, 32, 6, 2, 8, "paired", [50], whole(900)),
    (BF, 128, 28, 4, 32, "heads", [64, 20], [((5, 300), (380, 1)), ((37, 0), (130, 3))]),
    (HF, 128, 14, 2, 16, "slots", [19, 2, 4],
     [((100, 60), (0, 120)), ((0, 300), (40, 30)), ((200, 30), (190, 60))]),       # overlapping
    (BF, 64, 4, 4, 64, "heads", [3, 3, 3], [((10, -4), (70, 1)), ((127, 2), (0, 0)), ((0, 0), (0, 0))]),
    (BF, 128, 4, 1, 64, "heads", [2], whole(9000)),                                 # keys split over CTAs
    (HF, 128, 4, 2, 128, "slots", [300], whole(1300)),
    (BF, 128, 2, 2, 16, "heads", [1] * 200, whole(*[(i * 37) % 400 for i in range(200)])),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: str(c)[:90])
def test_attn(case):
    run_attn(*case)


@pytest.mark.parametrize("case", [ATTN[2], ATTN[6], ATTN[10], ATTN[15]], ids=lambda c: str(c)[:60])
@pytest.mark.parametrize("mask", ["causal", "blocks", "random", "nothing"])
def test_attn_row_limits(case, mask):
    segs, rows = case[7], case[6]
    end = [max(a + n for a, n in sg) for sg in segs]
    rng = random.Random(5)
    f = {"causal": lambda s, j: end[s] - rows[s] + j + 1,
         "blocks": lambda s, j: min(end[s], ((end[s] - rows[s] + j) // 32 + 1) * 32),
         "random": lambda s, j: rng.choice([0, 1, -7, 2 ** 31 - 1, rng.randint(0, end[s] + 3)]),
         "nothing": lambda s, j: 0}[mask]
    run_attn(*case, limit=f)


@pytest.mark.parametrize("case", [
    (BF, 128, 28, 4, 16, "heads", [1, 3, 2], whole(300, 129, 128)),       # 32-row tiles
    (HF, 128, 8, 8, 64, "slots", [40, 100, 33], whole(300, 700, 64)),      # 128-row tiles
    (BF, 64, 8, 2, 256, "heads", [90, 300], whole(900, 400)),              # several tiles
], ids=lambda c: str(c)[:60])
def test_slots_beyond_all_limits_hold_anything(case):
    lens = [sg[0][1] for sg in case[7]]
    for back in (1, 100):       # the last key seen is `back` before the segment's end
        run_attn(*case, limit=lambda s, j: lens[s] - back - j % 3, seen_only=True)
    run_attn(*case, limit=lambda s, j: 0 if s == 1 else 5, seen_only=True)
    n = len(lens)
    run_attn(*case, limit=lambda s, j: lens[s] - 7 * (s + 1) - j % 2, seen_only=True,
             groups=([0, n - 1, n], [70, 0]))


def test_attn_scale_and_large_scores():
    """Scores of several hundred: the running maximum has to carry them."""
    run_attn(*ATTN[3], scale=0.5, spread=20.0)
    run_attn(*ATTN[14], scale=0.3, spread=20.0)


SHARED = [  # dtype, D, Hq, Hkv, page, layout, rows, own segments, (first sequences, prefix lengths)
    (BF, 128, 28, 4, 16, "heads", [1] * 6, whole(1, 40, 16, 300, 0, 17), ([0, 6], [500])),
    (HF, 128, 32, 32, 64, "slots", [32, 7, 32], whole(32, 100, 64), ([0, 3], [130])),
    (BF, 64, 8, 2, 32, "paired", [5, 0, 70, 3, 9], whole(20, 0, 100, 33, 0), ([1, 3, 3, 5], [77, 50, 1])),
    (HF, 32, 4, 4, 8, "padded", [8, 8, 8, 8], whole(8, 0, 8, 130), ([0, 2, 4], [0, 257])),
    (BF, 128, 7, 1, 128, "heads", [1, 1, 1, 1, 1], whole(0, 0, 0, 0, 0), ([0, 2, 4], [9000, 3])),
    (HF, 128, 14, 2, 16, "heads", [40] * 9, whole(*range(40, 400, 40)), ([0, 9], [1000])),
    # one query tile spans more sequences than a warp has lanes, some of them without rows
    (BF, 64, 2, 2, 16, "heads", [1 if i % 4 else 0 for i in range(200)],
     whole(*[(i * 7) % 41 for i in range(200)]), ([3, 190], [300])),
    (HF, 32, 3, 3, 8, "slots", [2] * 150, whole(*[i % 19 for i in range(150)]), ([0, 150], [129])),
    # every kind of sequence and group in one batch
    (BF, 128, 8, 2, 32, "heads", [1, 70, 0, 33, 1, 1, 200, 5], whole(300, 70, 50, 0, 1, 129, 700, 5),
     ([1, 2, 2, 5, 7], [128, 90, 1, 640])),
    (HF, 64, 64, 1, 64, "padded", [1, 3, 2], whole(9, 3, 200), ([0, 2, 3], [64, 65])),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: str(c)[:90])
def test_shared_prefix(case):
    run_attn(*case[:8], groups=case[8])


def test_many_sequences_and_groups():
    """More sequences than the threads that plan the work, in hundreds of groups."""
    n = 1000
    run_attn(BF, 32, 2, 1, 8, "heads", [(i * 5) % 3 for i in range(n)], whole(*[(i * 13) % 30 for i in range(n)]))
    run_attn(HF, 32, 2, 1, 8, "slots", [1 if i % 9 else 0 for i in range(n)], whole(*[i % 12 for i in range(n)]),
             groups=([min(3 * i + i % 2, n) for i in range(331)], [(i * 11) % 50 for i in range(330)]))


def test_first_call_may_be_captured():
    """In a process of its own: the first attention of all is a captured one."""
    import subprocess
    import sys

    from tests.conftest import ROOT
    code = ("import torch, sys; sys.path.insert(0, %r)\n"
            "from tests.test_gpu_paged import *\nfrom tests.test_gpu_paged import _gen\n"
            "g = _gen(1); pool = make_pool(g, 4, 2, 16, 64, BF, 'heads'); kv = make_kv(pool, 4, 3)\n"
            "q = torch.randn(3, 4, 64, generator=g).to(BF).to(DEV); out = torch.zeros_like(q)\n"
            "a = (q, ints([0, 3]), ints([[2, 0]]), ints(whole(20)))\n"
            "gr = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(gr):\n    kv.attn(*a, out=out)\n"
            "gr.replay(); torch.cuda.synchronize()\n"
            "check_rows(out, R.attention(host(pool), q.cpu(), [0, 3], a[2].cpu(), whole(20)))\n" % ROOT)
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_follow_their_pages_device_stream():
    """Back-to-back calls on a side stream see what was queued there before them."""
    g = _gen(31)
    pool = make_pool(g, 8, 2, 16, 64, BF, "heads")
    kv = make_kv(pool, 4, 4)
    x = torch.randn(4, 8, 64, generator=g).to(BF)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        d = x.pin_memory().to(DEV, non_blocking=True)
        q = kv.append(d[:, 4:6], d[:, 6:], ints([0, 4]), ints([[5, 1]]), ints([14]), q=d[:, :4], rope_theta=1e4)
        out = kv.attn(q, ints([0, 4]), ints([[5, 1]]), ints(whole(18)))
        assert kv.device_status() == 0      # waits for the stream
    ref = R.attention(host(pool), q.cpu(), [0, 4], torch.tensor([[5, 1]], dtype=torch.int32), whole(18))
    check_rows(out, ref)


def test_shared_prefix_row_limits_count_own_positions():
    for c in (SHARED[1], SHARED[5], SHARED[8]):
        run_attn(*c[:8], groups=c[8], limit=lambda s, j: j)


def test_bad_pages_read_as_zeros():
    g = _gen(9)
    pool = make_pool(g, 5, 2, 16, 64, BF, "heads")
    kv = make_kv(pool, 4, 6, 1)
    q = torch.randn(6, 4, 64, generator=g).to(BF).to(DEV)
    table = torch.tensor([[0, 99, 1], [-7, 5, 2], [3, 4, 2 ** 31 - 1]], dtype=torch.int32)
    segs, rs = whole(48, 40, 32), [0, 2, 4, 6]
    out = kv.attn(q, ints(rs), table.to(DEV), ints(segs))
    assert kv.device_status() == 4
    check_rows(out, R.attention(host(pool), q.cpu(), rs, table, segs))
    pt = torch.tensor([[4, -1]], dtype=torch.int32)
    out = kv.shared_prefix_attn(q, ints(rs), table.to(DEV), ints(segs), ints([0, 3]), pt.to(DEV), ints([20]))
    check_rows(out, R.attention(host(pool), q.cpu(), rs, table, segs, groups=([0, 3], pt, [20])))


def test_positions_outside_the_table_are_left_out():
    g = _gen(10)
    pool = make_pool(g, 5, 1, 16, 32, HF, "slots")
    q = torch.randn(4, 2, 32, generator=g).to(HF).to(DEV)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
    for segs in ([((0, 33), (0, 0)), ((-3, 10), (0, 0))], [((0, 2 ** 31 - 1), (0, 0)), ((2 ** 31 - 1, 2 ** 31 - 1), (4, 4))]):
        kv = make_kv(pool, 2, 4, 1)
        out = kv.attn(q, ints([0, 2, 4]), table.to(DEV), ints(segs))
        assert kv.device_status() == 4
        check_rows(out, R.attention(host(pool), q.cpu(), [0, 2, 4], table, segs, dtype=HF))
    kv = make_kv(pool, 2, 4, 1)
    out = kv.shared_prefix_attn(q, ints([0, 2, 4]), table.to(DEV), ints(whole(3, 4)), ints([0, 2]), ints([[4]]),
                                ints([2 ** 31 - 1]))
    assert kv.device_status() == 4
    check_rows(out, R.attention(host(pool), q.cpu(), [0, 2, 4], table, whole(3, 4), dtype=HF,
                                groups=([0, 2], torch.tensor([[4]], dtype=torch.int32), [16])))


def test_any_row_start_stays_in_bounds():
    g = _gen(11)
    pool = make_pool(g, 4, 1, 16, 64, BF, "heads")
    kv = make_kv(pool, 2, 8, 2)
    q = torch.randn(8, 2, 64, generator=g).to(BF).to(DEV)
    for rs in ([-5, 3, 100], [8, 4, 0], [2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 1]):
        kv.attn(q, ints(rs), ints([[0, 1], [2, 3]]), ints(whole(20, 32)))
        for gs in ([0, 1, 2], [-4, 7, 1], [2 ** 31 - 1, -(2 ** 31), 5]):
            kv.shared_prefix_attn(q, ints(rs), ints([[0, 1], [2, 3]]), ints(whole(20, 32)), ints(gs),
                                  ints([[3], [1]]), ints([9, -4]))
    torch.cuda.synchronize()


def test_pages_beyond_32_bit_offsets():
    """Pages 2^31 elements apart: the last one starts past element 2^32."""
    ensure_lib()
    g = _gen(12)
    stride = 2 ** 31
    flat = [torch.empty(2 * stride + 2 * 16 * 64, dtype=BF, device=DEV) for _ in range(2)]
    pool = [x.as_strided((3, 2, 16, 64), (stride, 16 * 64, 64, 1)) for x in flat]
    for x in pool:
        x.copy_(torch.randn(3, 2, 16, 64, generator=g).to(BF))
    kv = make_kv(pool, 4, 5)
    x = torch.randn(5, 8, 64, generator=g).to(BF).to(DEV)
    table = torch.tensor([[1, 2, 0]], dtype=torch.int32)
    q = kv.append(x[:, 4:6], x[:, 6:], ints([0, 5]), table.to(DEV), ints([20]), q=x[:, :4])
    ps = host(pool)
    assert torch.equal(ps.k[2, :, 4:9].transpose(0, 1), x[:, 4:6].cpu().to(R.F64))
    assert torch.equal(ps.v[2, :, 4:9].transpose(0, 1), x[:, 6:].cpu().to(R.F64))
    segs = whole(48)
    out = kv.attn(q, ints([0, 5]), table.to(DEV), ints(segs))
    check_rows(out, R.attention(ps, q.cpu(), [0, 5], table, segs))


# ------------------------------------------------------------------ as they are used
def test_serving_run_matches_the_contiguous_cache():
    """A prompt enters once, two samples of it decode a block each: their pages and the shared
    prefix give what dllm_block_attn gives over contiguous copies of the same keys."""
    import ctypes as C

    from diffusion_decoding_step_b200 import abi
    from diffusion_decoding_step_b200 import workload as wl
    from diffusion_decoding_step_b200.runtime import make_config, workspace_bytes
    from tests.gpu_util import ptr, stream
    g = _gen(21)
    hq, hkv, D, ps, P, B = 28, 4, 128, 16, 200, 32
    pool = make_pool(g, 40, hkv, ps, D, BF, "heads")
    order = torch.randperm(40, generator=g).to(torch.int32)
    ptab, at = make_tables([P], ps, order)
    tab, at = make_tables([B, B], ps, order, at)
    kv = make_kv(pool, hq, P, 1)
    prompt = torch.randn(P, hq + 2 * hkv, D, generator=g).to(BF).to(DEV)
    kv.append(prompt[:, hq:hq + hkv], prompt[:, hq + hkv:], ints([0, P]), ptab.to(DEV), ints([0]),
              rope_theta=1e6)
    rows = torch.randn(2 * B, hq + 2 * hkv, D, generator=g).to(BF).to(DEV)
    rs = ints([0, B, 2 * B])
    q = kv.append(rows[:, hq:hq + hkv], rows[:, hq + hkv:], rs, tab.to(DEV), ints([0, 0]),
                  q=rows[:, :hq], rope_theta=1e6, rope_shift=ints([P, P]))
    out = kv.shared_prefix_attn(q, rs, tab.to(DEV), ints(whole(B, B)), ints([0, 2]), ptab.to(DEV), ints([P]))
    assert P % ps == 8  # the prefix ends inside a page
    pages = host(pool)  # and the same keys in the contiguous cache
    w = wl.Workload("t", batch=2, n_layers=1, hidden=512, n_q_heads=hq, n_kv_heads=hkv, head_dim=D,
                    vocab=1024, prompt_len=P + 24, gen_len=B, block=B)
    S = w.seq_len
    kc = torch.zeros(1, 2, hkv, S, D, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    for i in range(2):
        for cache, x in ((kc, pages.k), (vc, pages.v)):
            pre = torch.cat([x[int(p)] for p in ptab[0]], 1)[:, :P]
            own = torch.cat([x[int(p)] for p in tab[i]], 1)[:, :B]
            cache[0, i, :, :P + B] = torch.cat([pre, own], 1).to(BF).to(DEV)
    cfg, n = make_config(w), workspace_bytes(w)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    abi.check(abi.dllm_workspace_init(C.byref(cfg), ptr(ws), n, stream()), "ws init")
    qb = q.reshape(2, B, hq, D).transpose(1, 2).contiguous()
    want = torch.empty(2 * B, hq * D, dtype=BF, device=DEV)
    segs = ints(whole(P + B, P + B))
    abi.check(abi.dllm_block_attn(C.byref(cfg), 0, B, ptr(qb), ptr(kc), ptr(vc), ptr(segs), ptr(want),
                                  ptr(ws), n, stream()), "attn")
    torch.cuda.synchronize()
    assert kv.device_status() == 0
    ref = R.attention(pages, q.cpu(), [0, B, 2 * B], tab, whole(B, B), groups=([0, 2], ptab, [P]))
    check_rows(out, ref)
    check_rows(want.reshape(2 * B, hq, D), ref)


def test_captured_run_replays_with_new_contents():
    """Append and attention captured once; replays follow the row starts, positions, tables and
    lengths that the tensors hold then."""
    g = _gen(22)
    hq, hkv, D, ps, n = 8, 2, 64, 16, 6
    pool = make_pool(g, 64, hkv, ps, D, HF, "slots")
    kv = make_kv(pool, hq, n)
    x = torch.zeros(n, hq + 2 * hkv, D, dtype=HF, device=DEV)
    rs, pos = ints([0, 1, 2, 3]), ints([0, 0, 0])
    table = ints([[-1] * 20] * 3)
    segs = ints(whole(0, 0, 0))
    qo, out = torch.zeros(n, hq, D, dtype=HF, device=DEV), torch.zeros(n, hq, D, dtype=HF, device=DEV)

    def step():
        kv.append(x[:, hq:hq + hkv], x[:, hq + hkv:], rs, table, pos, q=x[:, :hq], q_out=qo, rope_theta=1e4)
        kv.attn(qo, rs, table, segs, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    order = torch.randperm(64, generator=g).to(torch.int32)
    for rows, lens in (([1, 1, 1], [5, 100, 300]), ([0, 4, 2], [0, 250, 17]), ([3, 0, 0], [129, 0, 0])):
        tab, _ = make_tables(lens, ps, order, width=20)
        x.copy_(torch.randn(x.shape, generator=g).to(HF))
        start = [sum(rows[:i]) for i in range(4)]
        rs.copy_(ints(start))
        pos.copy_(ints([b - a for a, b in zip(rows, lens)]))
        table.copy_(tab)
        segs.copy_(ints(whole(*lens)))
        graph.replay()
        torch.cuda.synchronize()
        ref = R.attention(host(pool), qo.cpu(), start, tab, whole(*lens), dtype=HF)
        assert len(ref) == sum(rows)
        check_rows(out, ref)
        for s in range(3):
            for j in range(rows[s]):
                p = lens[s] - rows[s] + j
                assert torch.equal(pool[1][int(tab[s, p // ps]), :, p % ps], x[start[s] + j, hq + hkv:])


def test_two_caches_on_two_streams():
    g = _gen(23)
    pool = make_pool(g, 300, 4, 64, 128, BF, "heads")
    order = torch.randperm(300, generator=g).to(torch.int32)
    tab, _ = make_tables([9000, 5000], 64, order)
    jobs = []
    for i in range(2):
        q = torch.randn(40, 28, 128, generator=g).to(BF).to(DEV)
        jobs.append((make_kv(pool, 28, 40), q, torch.cuda.Stream()))
    args = (ints([0, 20, 40]), tab.to(DEV), ints(whole(9000, 5000)))
    want = [kv.attn(q, *args) for kv, q, _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (kv, q, st) in enumerate(jobs):
            with torch.cuda.stream(st):
                got[i].append(kv.attn(q, *args))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o, want[i])


def test_arguments_are_checked():
    g = _gen(24)
    pool = make_pool(g, 4, 2, 16, 64, BF, "heads")
    kv = make_kv(pool, 4, 3, 1)
    from diffusion_decoding_step_b200.abi import DllmError
    from diffusion_decoding_step_b200.paged import PagedKV
    q = torch.zeros(3, 4, 64, dtype=BF, device=DEV)
    k = torch.zeros(3, 2, 64, dtype=BF, device=DEV)
    rs, tab, segs, pos = ints([0, 3]), ints([[0, 1]]), ints(whole(3)), ints([0])
    ok = kv.attn(q, rs, tab, segs)
    assert ok.shape == q.shape
    bad = [
        lambda: kv.attn(q.half(), rs, tab, segs),
        lambda: kv.attn(q[:, :3], rs, tab, segs),
        lambda: kv.attn(q.transpose(1, 2).contiguous().transpose(1, 2), rs, tab, segs),
        lambda: kv.attn(torch.zeros(4, 4, 64, dtype=BF, device=DEV), rs, tab, segs),
        lambda: kv.attn(q, rs.long(), tab, segs),
        lambda: kv.attn(q, rs, tab.cpu(), segs),
        lambda: kv.attn(q, rs, tab, segs[:, :1]),
        lambda: kv.attn(q, rs, tab, segs, row_limit=ints([1, 2])),
        lambda: kv.attn(q, rs, tab, segs, lse=torch.zeros(3, 3, device=DEV)),
        lambda: kv.attn(q, rs, tab, segs, out=q[:2]),
        lambda: kv.shared_prefix_attn(q, rs, tab, segs, ints([0, 1, 1]), ints([[2], [3]]), ints([4, 4])),
        lambda: kv.shared_prefix_attn(q, rs, tab, segs, None, None, None),
        lambda: kv.shared_prefix_attn(q, rs, tab, segs, ints([0, 1]), ints([[2]]), None),
        lambda: kv.attn(None, rs, tab, segs),
        lambda: kv.attn(q, [0, 3], tab, segs),
        lambda: kv.attn(q, rs, tab[0], segs),
        lambda: kv.append(k, k[:2], rs, tab, pos),
        lambda: kv.append(k, k, rs, tab, ints([0, 0])),
        lambda: kv.append(k, k, rs, tab, pos, q_out=q),
        lambda: PagedKV(pool[0], pool[1].float(), 4, 3),
        lambda: PagedKV(pool[0].float(), pool[1].float(), 4, 3),
        lambda: PagedKV(pool[0].transpose(2, 3), pool[1].transpose(2, 3), 4, 3),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    refused = [
        lambda: kv.attn(q, rs, tab, segs, out=q),
        lambda: kv.attn(q, rs, tab, segs, scale=-1.0),
        lambda: kv.attn(q, rs, tab, segs, scale=math.nan),
        lambda: kv.attn(q, rs, tab, segs, scale=3e38),
        lambda: kv.append(k, k, rs, tab, pos, rope_theta=math.inf),
        lambda: PagedKV(pool[0], pool[1], 3, 3),
        lambda: PagedKV(pool[0][:, :, :12], pool[1][:, :, :12], 4, 3),
        lambda: PagedKV(pool[0][..., :48], pool[1][..., :48], 4, 3),
    ]
    for i, f in enumerate(refused):
        with pytest.raises(DllmError):
            f()
            pytest.fail(f"call {i} was accepted")
    odd = torch.zeros(3 * 4 * 64 + 1, dtype=BF, device=DEV)[1:].view(3, 4, 64)  # not 16-byte aligned
    with pytest.raises(DllmError):
        kv.attn(odd, rs, tab, segs)
    assert kv.device_status() == 0
