"""Rows of the cache that a tile of queries does not see (later tokens of the same
chunk) have no part in its outputs, whatever they hold."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_gpu_paged import DEV, attend, cu_of, filled_cache, i32, tables

pytestmark = pytest.mark.gpu
HQ, HKV = 8, 2  # 32 tokens a tile


def bad_rows(kind, k, v, at):
    """The rows ``at`` of k and v, replaced."""
    if kind == "nan value":
        v[at, :, 5] = float("nan")
    elif kind == "inf value":
        v[at, :, 7] = float("inf")
    elif kind == "nan key":
        k[at, :, 3] = float("nan")
    else:
        k[at] *= 2.0 ** 40
        v[at] *= 2.0 ** 40


@pytest.mark.parametrize("kind", ["nan value", "inf value", "nan key", "large"])
@pytest.mark.parametrize("fmt,n_seq,chunk,before,n_splits", [
    ("bf16", 1, 300, 0, 1), ("bf16", 2, 300, 37, 1), ("bf16", 1, 300, 500, 3),
    ("e4m3", 1, 60, 0, 1), ("e4m3", 2, 60, 37, 2), ("nvfp4", 2, 60, 37, 1),  # converted on the chip
    ("e4m3", 1, 300, 0, 1), ("nvfp4", 1, 300, 37, 2),                        # widened first
    ("bf16", 30, 200, 0, 1), ("bf16", 30, 200, 37, 1), ("bf16", 30, 200, 300, 3),  # more tiles than SMs
    ("e4m3", 30, 200, 37, 1),
])
def test_later_tokens_do_not_reach_earlier_tiles(kind, fmt, n_seq, chunk, before, n_splits):
    g = np.random.default_rng(chunk + before)
    lens, total = [before + chunk] * n_seq, (before + chunk) * n_seq
    at = min(100, chunk - 20)  # the token of the bad row, in the same block as tiles before it
    tile = at - at % 32
    table, n_pages = tables(lens, 32, g)
    q = torch.from_numpy(g.standard_normal((chunk * n_seq, HQ, 128))).to(DEV, torch.bfloat16)
    k, v = (torch.from_numpy(g.standard_normal((total, HKV, 128))).to(DEV, torch.bfloat16)
            for _ in range(2))
    outs = []
    for bad in (False, True):
        if bad:
            for s in range(0, n_seq, 2):
                bad_rows(kind, k, v, s * (before + chunk) + before + at)
        kv = filled_cache(fmt, n_pages, 32, HKV)
        bs.attn_skip_kv_append(kv, k, v, cu_of(lens), i32(lens), table)
        q, out = attend(kv, table, [chunk] * n_seq, lens, HQ, [0.0] * n_seq, n_splits=n_splits, q=q)
        outs.append(out)
    (o0, l0, _), (o1, l1, _) = outs
    assert torch.isfinite(o0).all() and torch.isfinite(l0).all()
    for s in range(n_seq):
        rows = slice(s * chunk, s * chunk + (tile if s % 2 == 0 else chunk))
        assert torch.equal(o1[rows], o0[rows]) and torch.equal(l1[rows], l0[rows]), f"sequence {s}"
        seen = slice(s * chunk + at, (s + 1) * chunk)
        if s % 2 == 0 and kind != "large":
            x = l1[seen] if kind == "nan key" else o1[seen] if fmt != "bf16" else \
                o1[seen][..., 5 if kind == "nan value" else 7]
            assert not torch.isfinite(x).any()
            if kind == "nan value":  # the weights do not depend on the values
                assert torch.equal(l1[seen], l0[seen]) or torch.isfinite(l1[seen]).all()
