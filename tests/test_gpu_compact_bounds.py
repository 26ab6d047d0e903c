"""attn_skip_kv_compact where some bounds are bad: the sequences with good ones move as if they
were alone, in place and into other pages, and the error is reported."""
import random

import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import DEV, host, i32, no_error, pools, reported, same

pytestmark = pytest.mark.gpu

BOUNDS = [
    [0, 5, 3, 8],                  # a sequence goes back: the first and the last share rows
    [0, 10, -5, 20, 30], [0, 10, 99, 20, 30], [0, 10, 5, 20, 2, 30],
    [20, 5, 10], [30, 0, 30], [0, 30, 0, 30, 0, 30],
    [3, 3, 1, 30], [-1, 0, 30], [0, 31], [30, 29, 28, 27],
    [0, 600, 300, 900, 100, 600],  # more rows than a CTA takes at a time
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("per_head", [True, False])
@pytest.mark.parametrize("n_layers,Hkv", [(1, 1), (3, 2)])
def test_good_sequences_among_bad_ones(fmt, in_place, per_head, n_layers, Hkv):
    ps = 16
    for number, cu in enumerate(BOUNDS):
        r = random.Random(number)
        n, total = len(cu) - 1, 30 if max(cu) < 100 else 900
        good = [s for s in range(n) if 0 <= cu[s] <= cu[s + 1] <= total]
        width = plain.up(total + 5, ps)
        ids = r.sample(range(2 * n * width), 2 * n * width)
        table = [[ids.pop() for _ in range(width)] for _ in range(n)]
        out = None if in_place else [[ids.pop() for _ in range(width)] for _ in range(n)]
        # Row c of the batch is number c - cu[s] of a sequence: positions of at least that (in place).
        keep = [[c + r.randint(0, 5) if in_place else r.randrange(total) for c in range(total)]
                for _ in range(Hkv if per_head else 1)]
        kv, parts = pools(fmt, n_layers, 2 * n * width, Hkv, ps, number)
        want = host(parts)
        for s in good:
            kept = [k[cu[s]:cu[s + 1]] for k in keep]
            want = [{m: plain.compact(x, kept if per_head else kept[0], [0, cu[s + 1] - cu[s]],
                                      [table[s]], ps, None, None if in_place else [out[s]])
                     for m, x in p.items()} for p in want]
        k = torch.tensor(keep if per_head else keep[0], dtype=torch.int32, device=DEV)
        bs.attn_skip_kv_compact(kv, k, i32(cu), i32(table), out_table=None if in_place else i32(out))
        reported()
        same(parts, want)
    no_error()


def test_bad_places_next_to_bad_bounds():
    """Rows of positions or pages out of range stay out of a good sequence next to a bad one too."""
    kv, parts = pools("e4m3", 1, 12, 1, 16, 4)
    before = host(parts)
    keep, table, out = [5, 40, -1, 17, 9], [[0, 99], [1, 2], [3, 4]], [[5, 6], [7, 8], [9, 10]]
    bs.attn_skip_kv_compact(kv, i32(keep), i32([0, 5, 2, 5]), i32(table), out_table=i32(out))
    reported()
    x = [{m: plain.compact(x, [5], [0, 1], [table[0]], 16, None, [out[0]]) for m, x in p.items()}
         for p in before]
    x = [{m: plain.compact(x, [9], [0, 1], [table[0]], 16, [4], [out[0]]) for m, x in p.items()}
         for p in x]
    x = [{m: plain.compact(x, [17, 9], [0, 2], [table[2]], 16, [1], [out[2]]) for m, x in p.items()}
         for p in x]
    same(parts, x)
