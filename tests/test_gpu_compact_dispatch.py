"""Rows compacted in place by every group of threads that takes them: a warp, a CTA, rings of one
CTA or of a cluster, one launch or several; the batches are checked to go the way they are for."""
import random

import numpy as np
import pytest

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import host, i32, no_error, pools, same

pytestmark = pytest.mark.gpu
ROW = {"bf16": 256, "e4m3": 128, "nvfp4": 64}


def launches(fmt, n_layers, Hkv, counts):
    """The launches of a call: who takes the rows of which counts."""
    total, n = sum(counts), len(counts)
    units, mean, few = n_layers * n * Hkv, total // n, 12288 // (2 * ROW[fmt])

    def ring(at_once, kept):
        cta = 1
        while cta < 16 and 2 * at_once * cta < 128:
            cta *= 2
        clusters = min(2 * units, 304 // cta) if kept else 2 * units
        return f"ring{cta}", clusters

    out = []
    all_few = total <= 4 * few
    if not (units >= 608 and (all_few or (units >= 2048 and mean <= few // 2))):
        few = 0
    if few:
        out.append(("warp", None))
        if all_few:
            return out
    if (units < 160 and mean > 256) or (units < 320 and mean > 1024):
        return out + [ring(units, few)]
    out.append(("cta", None))
    if n_layers * Hkv <= 64 and total > 4096:
        out.append(ring(n_layers * Hkv, total // 2))
    return out


def check(fmt, n_layers, Hkv, ps, lengths, counts, keep_of, seed):
    r = random.Random(seed)
    per = [plain.up(x, ps) for x in lengths]
    ids, width = r.sample(range(sum(per)), sum(per)), max(per)
    table = [[ids.pop() for _ in range(p)] + [-1] * (width - p) for p in per]
    keep = [k for x, c in zip(lengths, counts) for k in keep_of(r, x, c)]
    cu = np.concatenate(([0], np.cumsum(counts))).tolist()
    kv, parts = pools(fmt, n_layers, sum(per), Hkv, ps, seed)
    before = host(parts)
    bs.attn_skip_kv_compact(kv, i32(keep), i32(cu), i32(table))
    no_error()
    some = [s for s, c in enumerate(counts) if c]  # (the plain form goes by sequences)
    same(parts, [{m: plain.compact(x, keep, cu, table, ps) if len(some) == len(counts) else
                  plain.compact(x, keep, [0] + [cu[s + 1] for s in some], [table[s] for s in some], ps)
                  for m, x in p.items()} for p in before])


def by_one(r, x, c):
    """Every row is overwritten by the next."""
    return range(x - c, x)


def scattered(r, x, c):
    """In any order, some twice, none before its own place."""
    return [r.randrange(j, x) if r.random() < 0.9 else j for j in range(c)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("keep_of", [by_one, scattered])
@pytest.mark.parametrize("n_layers,n,Hkv,cta", [(4, 4, 4, 1), (2, 4, 4, 2), (2, 2, 4, 4), (1, 2, 4, 8),
                                                (1, 1, 4, 16), (2, 1, 1, 16)])
def test_rings(fmt, n_layers, n, Hkv, cta, keep_of):
    lengths = [3001, 1300, 257, 600][:n]
    counts = [x - 1 for x in lengths]
    assert launches(fmt, n_layers, Hkv, counts) == [(f"ring{cta}", 2 * n_layers * n * Hkv)]
    check(fmt, n_layers, Hkv, 16, lengths, counts, keep_of, cta)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("keep_of", [by_one, scattered])
@pytest.mark.parametrize("n_layers,n,Hkv,way", [
    (16, 38, 4, [("cta", None), ("ring1", 304)]), (8, 19, 4, [("cta", None), ("ring2", 152)]),
    (4, 19, 4, [("cta", None), ("ring4", 76)]), (2, 57, 2, [("cta", None), ("ring16", 19)]),
    (2, 600, 4, [("warp", None), ("cta", None), ("ring8", 38)]),
])
def test_a_lone_long_sequence_goes_to_rings(fmt, n_layers, n, Hkv, way, keep_of):
    """Behind the others; where a layer's units are a multiple of the clusters, the long
    sequence's of all layers come to the same ones, one after another."""
    r = random.Random(n)
    lengths, lone = [r.randint(1, 6) for _ in range(n)], n // 2
    lengths[0], lengths[-1], lengths[lone] = 300, 40, 4301
    counts = [r.randint(0, x - 1) for x in lengths]
    counts[0], counts[-1], counts[lone] = 290, 39, 4300
    assert launches(fmt, n_layers, Hkv, counts) == way
    assert sum(c > sum(counts) // 2 for c in counts) == 1
    clusters = way[-1][1]
    if n < 600:
        assert n * Hkv * 2 % clusters == 0 and n_layers > 1
    check(fmt, n_layers, Hkv, 16, lengths, counts, keep_of, n)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("n_layers,n,Hkv,longest,way", [
    (8, 20, 4, 6, ["warp"]), (4, 160, 4, 30, ["warp", "cta"]), (2, 20, 4, 90, ["cta"]),
    (2, 40, 2, 2500, ["cta", "ring16"]),  # two of them: neither is more than half of all
])
def test_warps_and_ctas(fmt, n_layers, n, Hkv, longest, way):
    r = random.Random(n)
    lengths = [r.randint(1, 8) for _ in range(n)]
    counts = [r.randint(0, min(2, x - 1)) for x in lengths]
    for s in (3, 11):
        lengths[s], counts[s] = longest + 1, longest
    if way == ["warp", "cta"]:  # more rows than the warps take without looking
        for s in range(12, 24):
            lengths[s], counts[s] = 35, 34
    assert [w for w, _ in launches(fmt, n_layers, Hkv, counts)] == way
    if way == ["cta", "ring16"]:  # the rings find nothing to do
        assert max(counts) <= sum(counts) // 2
    check(fmt, n_layers, Hkv, 16, lengths, counts, scattered, n)
