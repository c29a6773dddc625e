"""The paged cache operators' refusals, and their 64-bit reference (no GPU)."""
import ctypes as C
import math

import pytest
import torch

from diffusion_decoding_step_b200 import abi, build
from tests import paged_ref as R

OK, INVALID, UNSUPPORTED, WORKSPACE = (abi.DLLM_OK, abi.DLLM_ERR_INVALID, abi.DLLM_ERR_UNSUPPORTED,
                                       abi.DLLM_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.lib()


D0 = 1 << 20   # aligned, never dereferenced


def pages(**kw):
    a = dict(k=D0, v=D0, page_stride=4 * 64 * 128, head_stride=64 * 128, slot_stride=128, n_pages=10,
             page_size=64, n_kv_heads=4, head_dim=128, type=0)
    a.update(kw)
    return C.byref(abi.dllm_kv_pages(**a))


def batch(**kw):
    a = dict(n_seqs=2, n_rows=5, max_pages=8, table_stride=8, row_start=D0, page_table=D0)
    a.update(kw)
    return C.byref(abi.dllm_paged_batch(**a))


def rows(**kw):
    a = dict(data=D0, row_stride=28 * 128, head_stride=128)
    a.update(kw)
    return C.byref(abi.dllm_rows(**a))


def groups(**kw):
    a = dict(n_groups=1, max_pages=4, table_stride=4, seq_start=D0, page_table=D0, len=D0)
    a.update(kw)
    return C.byref(abi.dllm_prefix_groups(**a))


def size(kv, hq=28, n=5):
    out = C.c_size_t(0)
    return abi.dllm_paged_workspace_size(kv, hq, n, C.byref(out)), out.value


def test_workspace_size(lib):
    st, least = size(pages())
    assert st == OK and least >= 4096
    assert size(pages(), n=2000)[1] >= size(pages(), n=18)[1] >= least
    assert size(pages(head_dim=96))[0] == UNSUPPORTED
    assert size(pages(page_size=48))[0] == UNSUPPORTED
    assert size(pages(page_size=4))[0] == UNSUPPORTED
    assert size(pages(page_size=1 << 17))[0] == UNSUPPORTED
    assert size(pages(page_size=0))[0] == INVALID
    assert size(pages(n_pages=0))[0] == INVALID
    assert size(pages(type=2))[0] == INVALID
    assert size(pages(), hq=27)[0] == INVALID
    assert size(pages(), hq=0)[0] == INVALID
    assert size(pages(n_kv_heads=1), hq=129)[0] == UNSUPPORTED
    assert size(pages(), n=0)[0] == INVALID
    assert size(pages(), n=1 << 24)[0] == UNSUPPORTED
    assert size(None)[0] == INVALID
    assert abi.dllm_paged_workspace_size(pages(), 28, 5, None) == INVALID
    assert abi.dllm_paged_workspace_init(None, 256, None) == INVALID
    assert abi.dllm_paged_workspace_init(D0 + 8, 256, None) == INVALID
    assert abi.dllm_paged_workspace_init(D0, 4095, None) == WORKSPACE


BAD_POOL = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=D0 + 8), INVALID),
            (dict(slot_stride=132), INVALID), (dict(slot_stride=64), INVALID), (dict(head_stride=0), INVALID),
            (dict(page_stride=1 << 39), INVALID), (dict(head_dim=16), UNSUPPORTED), (dict(n_kv_heads=0), INVALID)]
BAD_BATCH = [(dict(n_seqs=0), INVALID), (dict(n_seqs=1025), UNSUPPORTED), (dict(n_rows=0), INVALID),
             (dict(n_rows=1 << 24), UNSUPPORTED), (dict(max_pages=0), INVALID), (dict(table_stride=7), INVALID),
             (dict(max_pages=1 << 19, table_stride=1 << 19), UNSUPPORTED), (dict(row_start=None), INVALID),
             (dict(page_table=D0 + 2), INVALID)]
BAD_ROWS = [dict(data=None), dict(data=D0 + 2), dict(row_stride=28 * 128 + 4), dict(head_stride=64)]


def no_gpu():
    if torch.cuda.is_available():   # a regression would launch on the dummy pointers
        pytest.skip("dummy device pointers: runs only where no GPU is visible")


def append(kv=None, bt=None, hq=28, q=None, k=None, v=None, qo=None, pos=D0, shift=None, theta=1e4,
           status=None):
    return abi.dllm_paged_append(kv or pages(), bt or batch(), hq, q, k or rows(), v or rows(), qo, pos,
                                 shift, theta, status, None)


def test_append_refusals(lib):
    no_gpu()
    assert abi.dllm_paged_append(None, batch(), 0, None, rows(), rows(), None, D0, None, 0., None, None) == INVALID
    assert abi.dllm_paged_append(pages(), None, 0, None, rows(), rows(), None, D0, None, 0., None, None) == INVALID
    assert abi.dllm_paged_append(pages(), batch(), 0, None, None, rows(), None, D0, None, 0., None, None) == INVALID
    for kw, want in BAD_POOL:
        assert append(kv=pages(**kw)) == want, kw
    for kw, want in BAD_BATCH:
        assert append(bt=batch(**kw)) == want, kw
    for kw in BAD_ROWS:
        assert append(k=rows(**kw)) == INVALID, kw
        assert append(v=rows(**kw)) == INVALID, kw
        assert append(q=rows(**kw), qo=rows()) == INVALID, kw
        assert append(q=rows(), qo=rows(**kw)) == INVALID, kw
    assert append(q=rows(), qo=None) == INVALID
    assert append(q=rows(), qo=rows(), hq=27) == INVALID
    assert append(q=rows(), qo=rows(row_stride=36 * 128)) == INVALID   # in place, other strides
    assert append(pos=None) == INVALID
    assert append(pos=D0 + 1) == INVALID
    for theta in (math.nan, math.inf, -1.0):
        assert append(theta=theta) == INVALID


def test_attention_refusals(lib):
    no_gpu()
    n = size(pages())[1]

    def both(want, kv=None, bt=None, hq=28, segs=D0, lim=None, scale=0.0, q=None, out=None, lse=None,
             ws=D0, short=0):
        kv, bt, q, out = kv or pages(), bt or batch(), q or rows(), out or rows(data=2 * D0)
        assert abi.dllm_paged_attn(kv, bt, hq, segs, lim, scale, q, out, lse, ws, n - short, None) == want
        assert abi.dllm_shared_prefix_attn(kv, bt, groups(), hq, segs, lim, scale, q, out, lse, ws, n - short,
                                           None) == want

    for kw, want in BAD_POOL:
        both(want, kv=pages(**kw))
    for kw, want in BAD_BATCH:
        both(want, bt=batch(**kw))
    for kw in BAD_ROWS:
        both(INVALID, q=rows(**kw))
        both(INVALID, out=rows(**kw))
    both(INVALID, out=rows())            # out is q
    both(INVALID, hq=30)
    both(INVALID, segs=None)
    both(INVALID, lim=D0 + 2)
    both(INVALID, lse=D0 + 1)
    for scale in (math.nan, math.inf, -0.5):
        both(INVALID, scale=scale)
    both(INVALID, ws=None)
    both(INVALID, ws=D0 + 16)
    both(WORKSPACE, short=1)
    for kw, want in [(dict(n_groups=0), INVALID), (dict(n_groups=1025), UNSUPPORTED), (dict(max_pages=0), INVALID),
                     (dict(table_stride=3), INVALID), (dict(seq_start=None), INVALID), (dict(len=D0 + 2), INVALID),
                     (dict(page_table=None), INVALID), (dict(max_pages=1 << 19, table_stride=1 << 19), UNSUPPORTED)]:
        assert abi.dllm_shared_prefix_attn(pages(), batch(), groups(**kw), 28, D0, None, 0.0, rows(),
                                           rows(data=2 * D0), None, D0, n, None) == want, kw
    assert abi.dllm_shared_prefix_attn(pages(), batch(), None, 28, D0, None, 0.0, rows(), rows(data=2 * D0), None,
                                       D0, n, None) == INVALID


def test_paged_kv_wants_gpu_pages(lib):
    from diffusion_decoding_step_b200.paged import PagedKV
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        PagedKV(k, k.clone(), 4, 8)
    with pytest.raises(ValueError):
        PagedKV(k, k[:3], 4, 8)


# ------------------------------------------------------------------ the reference itself
def test_reference_rotation_keeps_lengths_and_relative_angles():
    x = torch.randn(1, 2, 64, dtype=R.F64)
    y = torch.randn(1, 2, 64, dtype=R.F64)
    at = lambda v, p: R.rotate(v, torch.tensor([p]), 1e4)  # noqa: E731
    assert torch.allclose(at(x, 17).square().sum(-1), x.square().sum(-1))
    assert torch.allclose((at(x, 17) * at(y, 12)).sum(-1), (at(x, 905) * at(y, 900)).sum(-1))
    assert torch.equal(at(x, 0), x)


def test_reference_attention_by_hand():
    """Two keys of equal score average their values; a bad page counts as a zero key."""
    k = torch.zeros(2, 1, 8, 32, dtype=R.F64)
    v = torch.zeros_like(k)
    v[0, 0, 0], v[0, 0, 1], v[1, 0, 0] = 1.0, 3.0, 8.0
    q = torch.randn(1, 1, 32)
    p = R.Pages(k, v)
    table = torch.tensor([[0, 9, 1]], dtype=torch.int32)
    get = lambda segs, **kw: R.attention(p, q, [0, 1], table, [segs], **kw)[0]  # noqa: E731
    out, lse, _, _ = get(((0, 2), (0, 0)))
    assert torch.allclose(out, torch.full_like(out, 2.0)) and math.isclose(lse[0], math.log(2))
    out, lse, _, _ = get(((0, 1), (8, 3)))
    assert torch.allclose(out, torch.full_like(out, 0.25)) and math.isclose(lse[0], math.log(4))
    out, lse, _, _ = get(((0, 2), (1, 1)), row_limit=[1])
    assert torch.allclose(out, torch.ones_like(out)) and lse[0] == 0
    out, lse, _, _ = get(((0, 2), (0, 0)), row_limit=[0])
    assert (out == 0).all() and lse[0] == -math.inf
    out, _, _, _ = get(((0, 0), (0, 0)), groups=([0, 1], torch.tensor([[1]], dtype=torch.int32), [1]))
    assert torch.allclose(out, torch.full_like(out, 8.0))


def test_reference_shared_prefix_is_one_longer_sequence():
    g = torch.Generator().manual_seed(1)
    p = R.Pages(*(torch.randn(6, 2, 8, 32, generator=g, dtype=R.F64) for _ in range(2)))
    q = torch.randn(4, 4, 32, generator=g)
    pre, own = torch.tensor([[3, 1]], dtype=torch.int32), torch.tensor([[0, 2], [4, 5]], dtype=torch.int32)
    a = R.attention(p, q, [0, 2, 4], own, [((0, 11), (0, 0)), ((0, 5), (0, 0))], groups=([0, 2], pre, [16]))
    b = R.attention(p, q, [0, 2, 4], torch.cat([pre.expand(2, -1), own], 1),
                    [((0, 27), (0, 0)), ((0, 21), (0, 0))])
    for r in range(4):
        assert torch.allclose(a[r][0], b[r][0]) and torch.allclose(a[r][1], b[r][1])
