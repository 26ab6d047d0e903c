"""Attention over quantised pages whose rows lie far apart in scale: within a block,
and from block to block."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import paged_plain as plain
from tests.test_gpu_paged import DEV, attend, cu_of, filled_cache, i32, pool_rows, tables
from tests.test_gpu_paged_zero_values import planted

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("n", [1, 5, 20, 40])
@pytest.mark.parametrize("apart", [14, 15, 16, 18, 21, 24, 30])
def test_rows_of_one_block_far_apart(fmt, n, apart):
    """Every third row is 2^apart smaller than its neighbours.  Where a block is
    converted on the chip to tiles with one exponent E, its elements are off by at
    most 2^-25 2^E (E4M3) or 7 * 2^-25 2^E (NVFP4, which rounds the product of block
    scale and row factor, then that with the code): beyond the roundings of any
    call, a score moves by d = scale sum |q| times that, O by 2 d A + that, the LSE
    by d.  (At most 8 rows a tile: exact.)"""
    g, L, G = np.random.default_rng(apart), 300, 4
    table, n_pages = tables((L,), 16, g)
    kv = filled_cache(fmt, n_pages, 16, 1)
    x = g.standard_normal((2, L, 1, 128))
    # Some elements of a row much smaller than its largest: small block scales.
    x[:, :, :, 64:] *= 2.0 ** -9
    x[:, ::3] *= 2.0 ** -apart
    k, v = (torch.from_numpy(y).to(DEV, torch.float32) for y in x)
    bs.attn_skip_kv_append(kv, k, v, cu_of([L]), i32([L]), table)
    q, (o, lse, _) = attend(kv, table, (n,), (L,), G, [0.0])
    k, v = (pool_rows(kv, table, 0, L, w) for w in "kv")
    qs = q.double().cpu().numpy().reshape(n, 1, G, 128)
    scale = 128 ** -0.5
    r = plain.attend(qs, k, v, n, L, G, 0.0, True, scale, 3)
    off = 0.0 if n * G <= 8 else (1 if fmt == "e4m3" else 7) * 2.0 ** -25
    ek, ev = (2.0 ** (int(s.max()) - 127) for s in
              (getattr(kv, w + "_scale")[table[0].long()].where(
                  getattr(kv, w + "_scale")[table[0].long()] != 255, 0) for w in "kv"))
    d = 2.0 ** -17 * r["dots"] + scale * np.abs(qs).sum(-1) * off * ek
    tol = (2.0 ** -8 * 1.01 * (r["absv"] + np.abs(r["o"]))
           + (2 * d[..., None] + 2.0 ** -18) * r["absv"] + off * ev * 1.01)
    got = o.double().cpu().numpy().reshape(r["o"].shape)
    gl = lse.double().cpu().numpy().reshape(r["lse"].shape)
    assert (np.abs(got - r["o"]) <= tol).all()
    assert (np.abs(gl - r["lse"]) <= d + 2.0 ** -20 * (8 + np.abs(r["lse"]))).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("n", [1, 5, 20, 40])
@pytest.mark.parametrize("first", [0, 1, 2])
def test_the_largest_values_behind_the_smallest_weights(fmt, n, first):
    """Three blocks that bring the outputs as much: weights 1, 2^-60 and 2^-118, values
    2^-4, 2^56 and 2^114, in every order."""
    g = np.random.default_rng(5)
    L = 384
    b = (np.arange(L) // 128 + first) % 3
    s = np.log(2.0) * np.array([118.0, 58.0, 0.0])[b]
    v = g.standard_normal((L, 128)) * np.exp2(np.array([-4.0, 56.0, 114.0])[b])[:, None]
    planted(fmt, s, v, n, 1, G=1)
