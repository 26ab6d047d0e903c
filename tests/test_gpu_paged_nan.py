"""A NaN in a key or a query shows in the outputs, also where a threshold skips
blocks and where the keys are split."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_gpu_paged import DEV, FORMATS, attend, cu_of, filled_cache, i32, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,n_seq,chunk,L,Hq,n_splits", [
    *((f, 2, 1, 900, 8, 1) for f in FORMATS),       # 4 rows
    *((f, 2, 5, 900, 8, 1) for f in FORMATS),       # 20 rows
    *((f, 2, 20, 900, 8, 1) for f in FORMATS),      # 80 rows
    *((f, 2, 60, 900, 8, 2) for f in FORMATS),      # two tiles
    *((f, 2, 300, 1200, 8, 1) for f in FORMATS),    # many, widened
    ("bf16", 100, 1, 900, 8, 1), ("bf16", 100, 2, 900, 8, 2),   # more pieces than SMs
    ("e4m3", 100, 1, 900, 8, 2), ("nvfp4", 100, 1, 900, 8, 2),
    ("bf16", 30, 200, 900, 8, 1), ("bf16", 30, 200, 900, 8, 2),
])
def test_a_nan_key_is_not_skipped(fmt, n_seq, chunk, L, Hq, n_splits):
    """The first key has the weight and every later block falls below the threshold;
    one of them, of every other sequence, holds a NaN key."""
    Hkv, at, lam = 2, 300, 0.5
    g = np.random.default_rng(5)
    lens = [L] * n_seq
    table, n_pages = tables(lens, 32, g)
    kv = filled_cache(fmt, n_pages, 32, Hkv)
    k = torch.zeros(n_seq, L, Hkv, 128, device=DEV)
    k[..., 0] = torch.from_numpy(g.uniform(0, 1, (n_seq, L, Hkv))).to(DEV)
    nb = -(-L // 128)
    bps = -(-nb // n_splits)
    for first in range(0, nb, bps):
        k[:, first * 128, :, 0] = 20.0
    k[::2, at, :, 64] = float("nan")
    v = torch.from_numpy(g.standard_normal((n_seq * L, Hkv, 128))).to(DEV, torch.float32)
    bs.attn_skip_kv_append(kv, k.view(-1, Hkv, 128), v, cu_of(lens), i32(lens), table)
    q = torch.zeros(n_seq * chunk, Hq, 128, device=DEV)
    q[..., 0] = 1.0
    q, (o, lse, bits) = attend(kv, table, [chunk] * n_seq, lens, Hq, [lam] * n_seq, True, n_splits,
                               q=q.to(torch.bfloat16), scale=1.0)
    o, lse = o.view(n_seq, chunk, Hq, 128), lse.view(n_seq, chunk, Hq)
    assert torch.isnan(o[::2]).all() and torch.isnan(lse[::2]).all()
    assert torch.isfinite(o[1::2]).all() and torch.isfinite(lse[1::2]).all()
    b = bs.unpack_bits(bits, bps).numpy()  # [n_seq, Hkv, tiles, splits, bps]
    for s in range(n_seq):
        for t in range(b.shape[2]):
            seen = -(-(L - chunk + min(chunk, 32 * (t + 1))) // 128)
            for j in range(seen):
                # The first block of a split is kept, and in the split with the NaN
                # its block and all behind it, as its maximum is NaN from there on.
                kept = j % bps == 0 or (s % 2 == 0 and j >= at // 128 and j // bps == at // 128 // bps)
                assert (b[s, :, t, j // bps, j % bps] == (not kept)).all(), (s, t, j)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 6, 20, 60, 300])
@pytest.mark.parametrize("n_splits", [1, 3])
def test_a_nan_query_has_a_nan_lse(fmt, n, n_splits):
    g = np.random.default_rng(n)
    L, Hkv, Hq = 900, 2, 8
    table, n_pages = tables((L,), 32, g)
    kv = filled_cache(fmt, n_pages, 32, Hkv)
    k, v = (torch.from_numpy(g.standard_normal((L, Hkv, 128))).to(DEV, torch.bfloat16)
            for _ in range(2))
    bs.attn_skip_kv_append(kv, k, v, cu_of([L]), i32([L]), table)
    q = torch.from_numpy(g.standard_normal((n, Hq, 128))).to(DEV, torch.bfloat16)
    bad = q.clone()
    bad[n // 2, 3, 17] = float("nan")
    _, (o, lse, _) = attend(kv, table, (n,), (L,), Hq, [0.0], n_splits=n_splits, q=bad)
    _, (o0, l0, _) = attend(kv, table, (n,), (L,), Hq, [0.0], n_splits=n_splits, q=q)
    assert torch.isnan(o[n // 2, 3]).all() and torch.isnan(lse[n // 2, 3])
    here = torch.ones(n, Hq, dtype=torch.bool, device=DEV)
    here[n // 2, 3] = False
    assert torch.equal(o[here], o0[here]) and torch.equal(lse[here], l0[here])
