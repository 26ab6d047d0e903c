"""Paged attention where the values say little about the weights: rows of zeros,
and rows whose scales lie far apart.  The row sum and the LSE belong to the
scores alone, whatever the values' exponents are."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_gpu_paged import DEV, FORMATS, attend, check, cu_of, filled_cache, i32, tables

pytestmark = pytest.mark.gpu
LN2 = math.log(2.0)
# Tokens of 4 heads: 4, 20 and 80 rows of one tile, two tiles.
TOKENS = (1, 5, 20, 40)


def planted(fmt, scores, values, n, n_splits, lam=0.0, G=4):
    """One sequence whose key c scores scores[c] (nats, about: keys are stored in
    ``fmt``) with every query, and whose values are given; checked."""
    L = len(scores)
    table, n_pages = tables((L,), 64, np.random.default_rng(L))
    kv = filled_cache(fmt, n_pages, 64, 1)
    k = torch.zeros(L, 1, 128, device=DEV)
    k[:, 0, 0] = torch.as_tensor(scores, dtype=torch.float32, device=DEV)
    v = torch.as_tensor(values, dtype=torch.float32, device=DEV).view(L, 1, 128)
    bs.attn_skip_kv_append(kv, k, v, cu_of([L]), i32([L]), table)
    q = torch.zeros(n, G, 128, device=DEV)
    q[:, :, 0] = 1.0 - torch.arange(G, device=DEV) / 16
    q, out = attend(kv, table, (n,), (L,), G, [lam], False, n_splits, q=q.to(torch.bfloat16), scale=1.0)
    check(kv, table, (n,), (L,), G, [lam], q, out, False, n_splits, scale=1.0)
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("n_splits", [1, 3])
@pytest.mark.parametrize("size,gap,L", [(300.0, 17, 32768), (1.0, 24, 32768), (5000.0, 20, 4096)])
def test_thousands_of_zero_values_below_one_key(fmt, n, n_splits, size, gap, L):
    g = np.random.default_rng(L)
    at = L // 2 + 77
    s, v = np.full(L, 0.5), np.zeros((L, 128))
    s[at], v[at] = 0.5 + gap * LN2, size * g.uniform(-1, 1, 128)
    planted(fmt, s, v, n, n_splits)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("size,gap", [(300.0, 17), (5000.0, 20)])
def test_thousands_of_zero_values_with_a_threshold(fmt, size, gap):
    L, g = 8192, np.random.default_rng(1)
    s, v = np.full(L, 0.5), np.zeros((L, 128))
    s[5000], v[5000] = 0.5 + gap * LN2, size * g.uniform(-1, 1, 128)
    for n in TOKENS:
        planted(fmt, s, v, n, 2, lam=1e-9)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", TOKENS)
def test_no_value_but_zeros(fmt, n):
    """The first key's score is 7 log2 units below all others'."""
    s = np.full(20000, 5.0)
    s[0] = 0.0
    o, lse, _ = planted(fmt, s, np.zeros((20000, 128)), n, 1)
    assert (o == 0).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("n_splits", [1, 2])
def test_blocks_of_zero_values_beside_blocks_of_small_ones(fmt, n, n_splits):
    g = np.random.default_rng(2)
    s, v = g.uniform(0, 3, 700), g.standard_normal((700, 128)) * 2.0 ** -45
    for a in (0, 256, 512):  # every other block, with the larger weights
        v[a:a + 128] = 0
        s[a:a + 128] += 6
    planted(fmt, s, v, n, n_splits)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", TOKENS)
@pytest.mark.parametrize("first", [0, 1])
def test_values_of_scales_far_apart(fmt, n, first):
    """Blocks of values 2^160 apart: the small ones' weights count all the same."""
    g = np.random.default_rng(3)
    s, v = g.uniform(0, 3, 600), g.standard_normal((600, 128))
    v *= np.exp2(np.where((np.arange(600) // 128) % 2 == first, 80.0, -80.0))[:, None]
    planted(fmt, s, v, n, 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", TOKENS)
def test_a_large_value_behind_a_low_score(fmt, n):
    """Two blocks that bring the outputs as much, one by weight, one by value."""
    g = np.random.default_rng(4)
    s, v = np.full(512, 40.0), g.standard_normal((512, 128))
    s[128:256], s[300] = 0.0, 1.0
    v[128:256] *= 2.0 ** 58
    planted(fmt, s, v, n, 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 6, 20])
@pytest.mark.parametrize("n_splits", [1, 3])
def test_a_nan_value_row_leaves_the_lse(fmt, n, n_splits):
    """Outputs of the rows that see it are NaN, their LSE is that of the scores."""
    g = np.random.default_rng(n)
    L = 400
    table, n_pages = tables((L,), 16, g)
    q = torch.from_numpy(g.standard_normal((n, 8, 128))).to(DEV, torch.bfloat16)
    k, v = (torch.from_numpy(g.standard_normal((L, 2, 128))).to(DEV, torch.bfloat16)
            for _ in range(2))
    lses = []
    for bad in (False, True):
        if bad:
            v[200] = float("nan")
            v[128:256] *= 0 if n == 1 else 1  # the only value of its block that is not zero
        kv = filled_cache(fmt, n_pages, 16, 2)
        bs.attn_skip_kv_append(kv, k, v, cu_of([L]), i32([L]), table)
        _, (o, lse, _) = attend(kv, table, (n,), (L,), 8, [0.0], n_splits=n_splits, q=q)
        lses.append(lse)
        assert torch.isnan(o).all() == bad and torch.isnan(o).any() == bad
    assert (lses[0] - lses[1]).abs().max() <= 2.0 ** -16
