"""Row bounds of the paged-cache calls: rows of no sequence on either side of the
batch."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_gpu_paged import DEV, FORMATS, cache_of, filled_cache, i32, tables

pytestmark = pytest.mark.gpu


def pool(kv):
    return [x.view(torch.uint8) for x in (kv.k, kv.v, kv.k_scale, kv.v_scale, kv.k_bs, kv.v_bs)
            if x is not None]


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
