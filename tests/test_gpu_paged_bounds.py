"""Row bounds of the paged-cache calls: rows of no sequence on either side of the
batch, and bounds that are refused."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_gpu_paged import DEV, FORMATS, cache_of, filled_cache, i32, pool_rows, tables

pytestmark = pytest.mark.gpu


def pool(kv):
    return [x.view(torch.uint8) for x in (kv.k, kv.v, kv.k_scale, kv.v_scale, kv.k_bs, kv.v_bs)
            if x is not None]


def refused():
    with pytest.raises(bs.AttnSkipError) as e:
        bs.attn_skip_last_device_error()
    assert e.value.status == bs.ATTN_EINVAL
    bs.attn_skip_last_device_error()  # cleared


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hkv,n,first", [(2, 30, 1), (3, 40, 6), (8, 10000, 3), (8, 10000, 5)])
def test_rows_before_the_first_sequence_are_ignored(fmt, Hkv, n, first):
    """A slice of a larger batch's bounds: the sequences need not start at row 0."""
    g = np.random.default_rng(n)
    lens = [n - 20, 11]
    total, bounds = first + sum(lens) + 3, i32([first, first + lens[0], first + sum(lens)])
    table, n_pages = tables(lens, 64, g)
    kv, ref = filled_cache(fmt, n_pages, 64, Hkv), filled_cache(fmt, n_pages, 64, Hkv)
    x, y = (torch.randn(total, Hkv, 128, device=DEV).to(torch.bfloat16) for _ in range(2))
    sub = slice(first, first + sum(lens))
    bs.attn_skip_kv_append(kv, x, y, bounds, i32(lens), table)
    bs.attn_skip_last_device_error()
    bs.attn_skip_kv_append(ref, x[sub], y[sub], bounds - first, i32(lens), table)
    bs.attn_skip_last_device_error()
    assert all(torch.equal(a, b) for a, b in zip(pool(kv), pool(ref)))
    out = [torch.full((total, Hkv, 128), 7.0, device=DEV) for _ in range(2)]
    bs.attn_skip_kv_gather(kv, bounds, None, table, total, out=out)
    bs.attn_skip_last_device_error()
    want = bs.attn_skip_kv_gather(ref, bounds - first, None, table, sum(lens), torch.float32)
    for a, b in zip(out, want):
        assert torch.equal(a[sub], b)
        assert (a[:first] == 7.0).all() and (a[sub.stop:] == 7.0).all()


@pytest.mark.parametrize("n_splits", [1, 3])
@pytest.mark.parametrize("fmt,lens", [("bf16", (5, 300)), ("e4m3", (1, 1)), ("nvfp4", (40, 9))])
def test_attention_of_a_batch_that_starts_behind_row_0(fmt, lens, n_splits):
    kv, table = cache_of(fmt, (700, 400), 32, 2, 3)
    total, first = sum(lens) + 9, 4
    q = torch.randn(total, 8, 128, device=DEV).to(torch.bfloat16)
    cu, kl, lam = i32([first, first + lens[0], first + sum(lens)]), i32([700, 400]), torch.zeros(2, device=DEV)
    o, lse = torch.full_like(q, 3.0), torch.full((total, 8), 3.0, device=DEV)
    bs.attn_skip_chunk_paged(kv, q, cu, max(lens), kl, 700, table, lam, n_splits=n_splits, out=(o, lse, None))
    sub = slice(first, first + sum(lens))
    want = bs.attn_skip_chunk_paged(kv, q[sub], cu - first, max(lens), kl, 700, table, lam, n_splits=n_splits)
    bs.attn_skip_last_device_error()
    assert torch.equal(o[sub], want[0]) and torch.equal(lse[sub], want[1])
    for x in (o, lse):
        assert (x[:first] == 3.0).all() and (x[sub.stop:] == 3.0).all()


BAD = [[0, 9], [-1, 3], [5, 2], [2, 0], [8, 20], [0, 3, 2, 5], [0, 4, 100], [0, 2, -3, 8]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cu", BAD)
def test_append_refuses_bad_bounds(fmt, cu):
    """Reported, whether or not a row of the call falls into the bad sequence; of its
    rows none is written, nor is any byte but those of sound sequences."""
    Hkv, ps, n = 2, 16, len(cu) - 1
    kv = filled_cache(fmt, 2 * n, ps, Hkv)
    ref = filled_cache(fmt, 2 * n, ps, Hkv)
    table = torch.arange(2 * n, dtype=torch.int32, device=DEV).view(n, 2)
    x = torch.randn(8, Hkv, 128, device=DEV).to(torch.bfloat16)
    lens = i32([20] * n)
    bs.attn_skip_kv_append(kv, x, x, i32(cu), lens, table)
    refused()
    sound = [s for s in range(n) if 0 <= cu[s] <= cu[s + 1] <= 8]
    page = torch.zeros(2 * n, dtype=torch.bool, device=DEV)
    for s in sound:
        bs.attn_skip_kv_append(ref, x, x, i32(cu[s:s + 2]), lens[:1], table[s:s + 1].contiguous())
        bs.attn_skip_last_device_error()
        page[table[s].long()] = True
    for a, b in zip(pool(kv), pool(ref)):
        assert torch.equal(a[~page], b[~page])   # (b: as it was made)
    if len(sound) == n - 1 and cu[1:] == sorted(cu[1:]):  # no two sequences claim a row
        assert all(torch.equal(a, b) for a, b in zip(pool(kv), pool(ref)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_writes_nothing_for_bad_pages_and_lengths(fmt):
    Hkv, ps = 2, 16
    kv = filled_cache(fmt, 6, ps, Hkv)
    ref = filled_cache(fmt, 6, ps, Hkv)
    x, y = (torch.randn(10, Hkv, 128, device=DEV).to(torch.bfloat16) for _ in range(2))
    # Page ids out of range; lengths beyond the table and below 0; one sound sequence.
    table = torch.tensor([[6, 0], [-1, 0], [1, 2], [3, 4], [5, 5]], dtype=torch.int32, device=DEV)
    bs.attn_skip_kv_append(kv, x, y, i32([0, 1, 2, 3, 5, 8]), i32([1, 1, 33, 17, -1]), table)
    refused()
    bs.attn_skip_kv_append(ref, x[3:5], y[3:5], i32([0, 2]), i32([17]), table[3:4].contiguous())
    bs.attn_skip_last_device_error()
    assert all(torch.equal(a, b) for a, b in zip(pool(kv), pool(ref)))
    assert not torch.equal(kv.v.view(torch.uint8), filled_cache(fmt, 6, ps, Hkv).v.view(torch.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cu", BAD)
def test_gather_refuses_bad_bounds(fmt, cu):
    """Reported; rows of the bad sequence that the call has read as zeros."""
    n = len(cu) - 1
    kv, table = cache_of(fmt, [40] * n, 16, 2, 8)
    out = [torch.full((8, 2, 128), 7.0, device=DEV) for _ in range(2)]
    bs.attn_skip_kv_gather(kv, i32(cu), None, table, 8, out=out)
    refused()
    if cu == [0, 4, 100]:
        for which, x in zip("kv", out):
            np.testing.assert_array_equal(x[:4].double().cpu().numpy(), pool_rows(kv, table, 0, 4, which))
            assert (x[4:] == 0).all()
    if cu == [0, 9]:
        assert all((x == 0).all() for x in out)
