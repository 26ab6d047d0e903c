"""Large batches of short key ranges with thresholds: a few rows a tile, more pieces
than SMs, at most twelve blocks a piece."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import DEV, FORMATS, attend, batch, cache_of, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,longest,kinds,n_splits", [
    (100, 400, (1, 1, 2), 1),
    (100, 1500, (1,), 1),
    (60, 1400, (1, 2, 8), 3),
    (160, 900, (1, 3, 8), 2),
    (90, 130, (1, 5), 1),
])
def test_few_rows_over_short_ranges_skip(fmt, n, longest, kinds, n_splits):
    Hkv, G = 2, 4
    assert n * Hkv * n_splits > 152 and -(-(-(-longest // 128)) // n_splits) <= 12
    chunks, lens = batch(n, longest, n, kinds)
    lams = [(0.0, 0.3, 0.6)[s % 3] for s in range(n)]
    kv, table = cache_of(fmt, lens, 32, Hkv, n, sink=1.0)
    g = np.random.default_rng(n)
    q = torch.from_numpy(g.standard_normal((sum(chunks), Hkv * G, 128)) + 0.7).to(DEV, torch.bfloat16)
    for causal in (True, False):
        q, out = attend(kv, table, chunks, lens, Hkv * G, lams, causal, n_splits, q=q)
        skipped = check(kv, table, chunks, lens, Hkv * G, lams, q, out, causal, n_splits)
        assert skipped > 0 or longest < 256  # (there two keys of a block, at most)
        again = attend(kv, table, chunks, lens, Hkv * G, lams, causal, n_splits, q=q)[1]
        assert all(torch.equal(a, b) for a, b in zip(out, again))
