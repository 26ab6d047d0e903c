"""Page bookkeeping, moved pages and moved rows against plain implementations: whole
numbers and bytes, compared for equality over whole tables and pools."""
import random

import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x, device=DEV):
    return torch.tensor(np.asarray(x, dtype=np.int32), device=device)


def no_error():
    bs.attn_skip_last_device_error()


def reported():
    with pytest.raises(bs.AttnSkipError) as e:
        bs.attn_skip_last_device_error()
    assert e.value.status == bs.ATTN_EINVAL


# ------------------------------------------------------------------- reserve --
def batch(seed, n, ps, max_kv, n_pages, share=0.0, grow=9):
    """Tables of sequences of random lengths, some of them forks of the one before."""
    r = random.Random(seed)
    width = plain.up(max_kv, ps)
    free = r.sample(range(n_pages), n_pages)
    refs, table, old, new = [0] * n_pages, [], [], []
    for s in range(n):
        if s and r.random() < share:
            row, a = list(table[-1]), old[-1]
        else:
            a = r.choice((0, r.randint(0, max_kv), ps * r.randint(0, max_kv // ps)))
            a = min(a, len(free) * ps)
            k = plain.up(a, ps)
            row = [free.pop() for _ in range(k)] + [r.choice((-1, 7, 1 << 30)) for _ in range(width - k)]
        for p in row[:plain.up(a, ps)]:
            refs[p] += 1
        table.append(row)
        old.append(a)
        new.append(min(max_kv, a + r.choice((0, 1, r.randint(0, grow)))))
    return refs, table, old, new


def check_reserve(refs, table, old, new, ps, alias=False):
    want = plain.reserve(refs, table, old, new, ps)
    R, T, a, b = i32(refs), i32(table), i32(old), i32(new)
    if alias:
        out = (a, torch.empty_like(a), torch.empty_like(a))
        got = bs.attn_skip_pages_reserve(R, T, a, b, ps, out=out)
    else:
        got = bs.attn_skip_pages_reserve(R, T, a, b, ps)
    assert R.tolist() == want[0]
    assert T.tolist() == want[1]
    for x, y in zip(got, want[2:5]):
        assert x.tolist() == y
    (reported if want[5] else no_error)()
    return want


@pytest.mark.parametrize("n,ps,max_kv,n_pages,share,grow", [
    (1, 16, 40, 1, 0.0, 40), (1, 1, 3, 31, 0.0, 3), (2, 16, 100, 32, 0.5, 20), (5, 3, 50, 33, 0.5, 9),
    (7, 16, 300, 90, 0.4, 60), (64, 16, 500, 2500, 0.3, 4), (64, 16, 500, 1500, 0.3, 100),
    (100, 64, 900, 8192, 0.6, 200), (100, 64, 900, 8193, 0.6, 200), (33, 7, 100, 70000, 0.9, 5),
    (300, 16, 64, 300000, 0.2, 30), (1023, 16, 40, 4000, 0.7, 9), (1025, 32, 64, 1100, 0.9, 40),
    (8192, 16, 16, 8200, 0.5, 16),
])
def test_reserve(n, ps, max_kv, n_pages, share, grow):
    for seed in range(3):
        check_reserve(*batch(seed + n, n, ps, max_kv, n_pages, share, grow), ps, alias=seed == 1)


def test_reserve_goes_on_in_place_behind_one_that_does_not_fit():
    """The second needs no page: it grows, and the free pages stay free."""
    got = check_reserve([1, 0, 1, 0], [[0, -1, -1, -1], [2, -1, -1, -1]], [4, 2], [16, 3], 4)
    assert got[0] == [1, 0, 1, 0] and got[2] == [4, 3]


def test_reserve_one_page_shared_by_all():
    # Parallel samples of one prompt: all but the last copy its last page.
    for n, n_pages in ((2, 4), (500, 600), (500, 200), (3000, 9000)):
        refs = [0] * n_pages
        refs[1] = refs[n_pages - 1] = n
        table = [[n_pages - 1, 1, -1]] * n
        want = check_reserve(refs, table, [20] * n, [21 + 15 * (s % 2) for s in range(n)], 16)
        assert sum(x >= 0 for x in want[3]) == min(n - 1, sum(x >= 0 for x in want[3]))


def test_reserve_holders_outside_of_the_batch():
    # Four references, two sequences: both copy, the page keeps the two that are not here.
    check_reserve([0, 4, 0, 0], [[1], [1]], [3, 3], [4, 4], 4)


def test_reserve_the_largest_pool_and_every_page_free():
    n_pages = 1 << 20
    R = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    T = torch.full((3, 5000), -1, dtype=torch.int32, device=DEV)
    got, _, _ = bs.attn_skip_pages_reserve(R, T, i32([0, 0, 0]), i32([16 * 5000, 1, 16 * 4000]), 16)
    assert got.tolist() == [80000, 1, 64000]
    assert torch.equal(T[0], torch.arange(5000, dtype=torch.int32, device=DEV))
    assert T[1, 0] == 5000 and T[2, 3999] == 9000 and int(R.sum()) == 9001
    assert torch.equal(R[:9001], torch.ones(9001, dtype=torch.int32, device=DEV))
    # Only the highest pages free.
    R.fill_(1)
    R[-7:] = 0
    got, _, _ = bs.attn_skip_pages_reserve(R, T, i32([0, 0, 0]), i32([16 * 4, 16 * 4, 0]), 16)
    assert got.tolist() == [64, 0, 0]
    assert T[0, :4].tolist() == [n_pages - 7 + i for i in range(4)]
    no_error()


def test_reserve_bad_lengths_are_left_out_and_reported():
    refs, table = [1, 0, 0, 0, 2, 0], [[0, -1], [4, -1], [4, -1], [99, -1], [-5, -1]]
    for old, new in (([4, -1, 3, 0, 0], [5, 3, 4, 3, 4]), ([4, 3, 3, 0, 0], [3, 4, 4, 9, 8]),
                     ([4, 3, 3, 3, 2], [5, 4, 4, 4, 4]), ([0, 0, 0, 0, 0], [1 << 30, 0, 0, 0, 2])):
        assert check_reserve(refs, table, old, new, 4)[5]


# ---------------------------------------------------------------------- fork --
def check_fork(refs, table, old, new, ps, parent=None, n_new=None):
    width = len(table[0])
    before = None if parent is None else [[-9 - i] * width for i in range(len(parent))]
    want = plain.fork(refs, table, old, new, ps, parent, before)
    R, T = i32(refs), i32(table)
    got = bs.attn_skip_pages_fork(R, T, i32(old), i32(new), ps,
                                  parent=None if parent is None else i32(parent),
                                  out_table=None if parent is None else i32(before))
    assert R.tolist() == want[0]
    assert got.tolist() == want[1]
    assert T.tolist() == [list(r) for r in table]
    no_error()


@pytest.mark.parametrize("n,ps,max_kv,share", [
    (1, 16, 16, 0.0), (2, 1, 30, 0.5), (9, 16, 300, 0.4), (32, 16, 2500, 0.7), (40, 64, 20000, 0.2),
    (301, 32, 500, 0.5),
])
def test_fork(n, ps, max_kv, share):
    for seed in range(3):
        r = random.Random(seed)
        need = n * plain.up(max_kv, ps) + 3
        refs, table, old, _ = batch(seed, n, ps, max_kv, need, share)
        check_fork(refs, table, old, [r.choice((0, a, r.randint(0, a))) for a in old], ps)
        for m in (1, n, 2 * n + 1):
            parent = [r.choice((-1, d % n, r.randrange(n))) for d in range(m)]
            new = [0 if p < 0 else r.choice((old[p], old[p], r.randint(0, old[p]))) for p in parent]
            check_fork(refs, table, old, new, ps, parent)
        check_fork(refs, table, old, [old[0]] * (3 * n), ps, [0] * (3 * n))  # all follow the first
        check_fork(refs, table, old, [0] * n, ps, [-1] * n)  # the batch ends


@pytest.mark.parametrize("followers", [24, 25, 1300])
@pytest.mark.parametrize("shortest,longest", [(0, 2500), (700, 720), (1, 1025), (2499, 2500)])
def test_fork_many_followers_of_different_lengths(followers, shortest, longest):
    r = random.Random(followers + shortest)
    refs, table = [1] * 2500 + [3] * 5, [list(range(2500)), [2504] * 2500]
    parent = [0] * followers + [1, -1]
    r.shuffle(parent)
    new = [(0 if p < 0 else 1 if p else r.randint(shortest, longest)) for p in parent]
    check_fork(refs, table, [2500, 1], new, 1, parent)


def test_fork_makes_its_table():
    R, T = i32([1, 1, 0]), i32([[0, 1]])
    out = bs.attn_skip_pages_fork(R, T, i32([20]), i32([20, 3, 0]), 16, parent=i32([0, 0, -1]))
    assert out.tolist() == [[0, 1], [0, -1], [-1, -1]] and R.tolist() == [2, 1, 0]
    with pytest.raises(ValueError):
        bs.attn_skip_pages_fork(R, T, i32([20]), i32([20]), 16, out_table=T.clone())
    with pytest.raises(bs.AttnSkipError):
        bs.attn_skip_pages_fork(R, T, i32([20]), i32([20]), 16, parent=i32([0]), out_table=T)
    no_error()


def test_fork_bad_arguments_are_reported():
    def call(old, new, parent, table=((0, 1), (2, -1))):
        R = i32([1, 1, 1])
        out = bs.attn_skip_pages_fork(R, i32(table), i32(old), i32(new), 4,
                                      parent=None if parent is None else i32(parent))
        reported()
        return R.tolist(), out.tolist()
    # Parents out of range, or none with a length: empty sequences.
    assert call([8, 4], [8, 4], [0, 2]) == ([1, 1, 0], [[0, 1], [-1, -1]])
    assert call([8, 4], [8, 4], [0, -2]) == ([1, 1, 0], [[0, 1], [-1, -1]])
    assert call([8, 4], [8, 4], [0, -1]) == ([1, 1, 0], [[0, 1], [-1, -1]])
    # Lengths beyond the parent's, or negative: the nearest in range.
    assert call([8, 4], [8, 8], [0, 1]) == ([1, 1, 1], [[0, 1], [2, -1]])
    assert call([8, 4], [8, -1], [0, 1]) == ([1, 1, 0], [[0, 1], [-1, -1]])
    assert call([8, 4], [9, 4], None)[0] == [1, 1, 1]
    assert call([8, 4], [-3, 4], None)[0] == [0, 0, 1]
    # A cached length out of range counts as 0.
    assert call([9, 4], [8, 4], [0, 1]) == ([1, 1, 1], [[-1, -1], [2, -1]])
    assert call([-1, 4], [0, 4], None)[0] == [1, 1, 1]
    # Page ids out of range are not counted.
    assert call([8, 4], [8, 0], [0, 1], ((0, 3), (-1, 5))) == ([1, 1, 1], [[0, 3], [-1, -1]])


# --------------------------------------------------------- pools of all kinds --
def pool(fmt, n_pages, Hkv, ps, seed, together=False):
    """Random bytes in every part; ``together``: k and v of a page next to each other."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    width = {"bf16": 256, "e4m3": 128, "nvfp4": 64}[fmt]

    def u8(*shape):
        return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=g)

    if together:
        both = u8(n_pages, 2, Hkv, ps, width)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = u8(n_pages, Hkv, ps, width), u8(n_pages, Hkv, ps, width)
    parts = dict(k=k, v=v)
    if fmt != "bf16":
        parts.update(k_scale=u8(n_pages, Hkv, ps), v_scale=u8(n_pages, Hkv, ps))
    if fmt == "nvfp4":
        parts.update(k_bs=u8(n_pages, Hkv, ps, 8), v_bs=u8(n_pages, Hkv, ps, 8))
    kv = bs.PagedKV(fmt, **{n: x.view(torch.bfloat16) if fmt == "bf16" else x
                            for n, x in parts.items()})
    return kv, parts


def pools(fmt, n_layers, n_pages, Hkv, ps, seed, together=False):
    got = [pool(fmt, n_pages, Hkv, ps, seed * 1000 + i, together) for i in range(n_layers)]
    return bs.PagedLayers([kv for kv, _ in got]), [p for _, p in got]


def host(parts):
    return [{n: x.cpu().numpy().copy() for n, x in p.items()} for p in parts]


def same(parts, want):
    for p, w in zip(parts, want):
        for n, x in p.items():
            equal = bool((x.cpu().numpy() == w[n]).all())
            assert equal, n


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("n_layers,n_pages,Hkv,ps,n,together", [
    (1, 2, 1, 16, 1, False), (1, 9, 3, 16, 4, True), (2, 21, 8, 64, 9, False),
    (65, 7, 1, 32, 3, False), (3, 40, 2, 384, 19, True),
    (40, 41, 1, 16, 18, False), (40, 45, 3, 32, 20, True),  # by warps, by CTAs
    (1, 1500, 1, 16, 700, False),  # more entries than are listed at a time
])
def test_copy_pages(fmt, n_layers, n_pages, Hkv, ps, n, together):
    r = random.Random(n_pages)
    kv, parts = pools(fmt, n_layers, n_pages, Hkv, ps, 5, together)
    before = host(parts)
    order = r.sample(range(n_pages), n_pages)
    src, dst = [r.choice(order[n:]) for _ in range(n)], order[:n]  # (a page may be copied twice)
    src += [-1, 0, -1, 1]
    dst += [0, -1, -1, 1]
    bs.attn_skip_kv_copy_pages(kv, i32(src), i32(dst))
    no_error()
    keep = [i for i in range(len(src)) if src[i] >= 0 and dst[i] >= 0]
    same(parts, [{m: plain.copy_pages(x, [src[i] for i in keep], [dst[i] for i in keep])
                  for m, x in p.items()} for p in before])
    # A single cache; bad ids are left out and reported.
    now = host(parts)
    bs.attn_skip_kv_copy_pages(kv.caches[0], i32([n_pages, -2, 0, 0]), i32([0, 0, n_pages, -7]))
    reported()
    bs.attn_skip_kv_copy_pages(kv, i32([]), i32([]))
    no_error()
    for bad in (n_pages, -2):  # onto itself
        bs.attn_skip_kv_copy_pages(kv, i32([-1, bad]), i32([0, bad]))
        reported()
    same(parts, now)


def rows(seed, n, ps, max_kv, in_place, heads=0):
    """Tables, kept positions (their place in the sequence at least), starts."""
    r = random.Random(seed)
    L = [r.choice((1, max_kv, r.randint(1, max_kv))) for _ in range(n)]
    per = [plain.up(x, ps) for x in L]
    n_pages = 2 * sum(per) + 2
    ids = r.sample(range(n_pages), n_pages)
    width = max(per)
    table = [[ids.pop() for _ in range(p)] + [-1] * (width - p) for p in per]
    out = None if in_place else [[ids.pop() for _ in range(p)] + [1 << 30] * (width - p) for p in per]
    count = [r.choice((0, x, r.randint(0, x))) for x in L]
    start = [r.randint(0, x - c) for x, c in zip(L, count)]
    keep = []
    for _ in range(heads or 1):
        one = []
        for x, c, st in zip(L, count, start):
            one += (sorted(r.sample(range(st, x), c)) if in_place
                    else [r.randrange(x) for _ in range(c)])  # any order, twice the same
        keep.append(one)
    cu = np.concatenate(([0], np.cumsum(count))).tolist()
    return n_pages, table, out, (keep if heads else keep[0]), cu, start


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n_layers,n,Hkv,ps,max_kv,per_head,together", [
    (1, 1, 1, 16, 5, False, False), (2, 3, 2, 16, 70, True, False), (1, 2, 3, 64, 700, False, True),
    (65, 2, 1, 32, 40, False, False), (1, 1, 2, 128, 3001, True, False), (2, 40, 1, 16, 90, False, True),
])
def test_compact(fmt, in_place, n_layers, n, Hkv, ps, max_kv, per_head, together):
    for seed in range(2):
        n_pages, table, out, keep, cu, start = rows(seed + max_kv, n, ps, max_kv, in_place,
                                                    Hkv if per_head else 0)
        kv, parts = pools(fmt, n_layers, n_pages, Hkv, ps, seed, together)
        before = host(parts)
        if seed and in_place:
            start = None  # (kept positions are at least their number)
        k = torch.tensor(keep, dtype=torch.int32, device=DEV)
        bs.attn_skip_kv_compact(kv, k, i32(cu), i32(table), start=None if start is None else i32(start),
                                out_table=None if out is None else i32(out))
        no_error()
        same(parts, [{m: plain.compact(x, keep, cu, table, ps, start, out) for m, x in p.items()}
                     for p in before])


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_compact_moves_rows_by_one(fmt):
    """Every row is overwritten by the next: the order of loads and stores matters most."""
    L, ps = 5000, 16
    n_pages = plain.up(L, ps)
    table = [random.Random(3).sample(range(n_pages), n_pages)]
    for Hkv in (1, 4):
        kv, parts = pools(fmt, 2, n_pages, Hkv, ps, 1)
        before = host(parts)
        keep = list(range(1, L))
        bs.attn_skip_kv_compact(kv, i32(keep), i32([0, L - 1]), i32(table))
        no_error()
        same(parts, [{m: plain.compact(x, keep, [0, L - 1], table, ps) for m, x in p.items()}
                     for p in before])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_one_long_sequence_among_many(fmt, in_place):
    """Most sequences keep nothing or a few rows, one keeps thousands; kept positions in any
    order, some twice (in place at least at their own place)."""
    r, ps, n = random.Random(5), 32, 90
    L = [r.randint(1, 70) for _ in range(n)]
    L[17], L[60] = 4000, 200
    per = [plain.up(x, ps) for x in L]
    n_pages = 2 * sum(per)
    ids, width = r.sample(range(n_pages), n_pages), max(per)
    table = [[ids.pop() for _ in range(p)] + [-1] * (width - p) for p in per]
    out = None if in_place else [[ids.pop() for _ in range(p)] + [-1] * (width - p) for p in per]
    keep, cu = [], [0]
    for s, x in enumerate(L):
        c = r.randint(2500, 3000) if s == 17 else 100 if s == 60 else r.choice((0, 0, r.randint(0, x)))
        keep += [r.randrange(j, x) if r.random() < 0.9 else j for j in range(c)]
        cu.append(len(keep))
    assert cu[-1] < 64 * n
    kv, parts = pools(fmt, 2, n_pages, 2, ps, 3)
    before = host(parts)
    bs.attn_skip_kv_compact(kv, i32(keep), i32(cu), i32(table),
                            out_table=None if out is None else i32(out))
    no_error()
    same(parts, [{m: plain.compact(x, keep, cu, table, ps, None, out) for m, x in p.items()}
                 for p in before])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
@pytest.mark.parametrize("n_layers,n,longest", [(40, 16, 0), (64, 40, 0), (64, 40, 190), (5, 140, 60)])
def test_compact_paths_of_trees(fmt, n_layers, n, longest):
    """Many short moves behind the cached rows in many layers, in place; one may be long."""
    r, ps = random.Random(n), 16
    L = [r.randint(20, 60) for _ in range(n)]
    count = [r.choice((0, 1)) for _ in range(n)]
    if longest:
        L[7], count[7] = 2 * longest, longest
    per = [plain.up(x, ps) for x in L]
    ids, width = r.sample(range(sum(per)), sum(per)), max(per)
    table = [[ids.pop() for _ in range(p)] + [-1] * (width - p) for p in per]
    # Positions ascend from the start on, so that a kept one is at least its new one.
    start = [max(0, x - 2 * c - 1) for x, c in zip(L, count)]
    keep = [k for x, c, st in zip(L, count, start) for k in sorted(r.sample(range(st, x), c))]
    cu = np.concatenate(([0], np.cumsum(count))).tolist()
    kv, parts = pools(fmt, n_layers, sum(per), 1, ps, 6)
    before = host(parts)
    bs.attn_skip_kv_compact(kv, i32(keep), i32(cu), i32(table), start=i32(start))
    no_error()
    same(parts, [{m: plain.compact(x, keep, cu, table, ps, start) for m, x in p.items()}
                 for p in before])


def test_compact_leaves_rows_outside_the_sequences_alone_and_reports():
    kv, parts = pool("e4m3", 6, 2, 16, 9)
    before = host([parts])

    def call(keep, cu, table=((0, 1), (2, 3)), out=None, start=None):
        bs.attn_skip_kv_compact(kv, i32(keep), i32(cu), i32(table),
                                start=None if start is None else i32(start),
                                out_table=None if out is None else i32(out))

    # Entries of keep before the first sequence and behind the last are ignored.
    call([99, 5, 7, 99], [1, 2, 3])
    no_error()
    want = [{m: plain.compact(x, [99, 5, 7, 99], [1, 2, 3], [[0, 1], [2, 3]], 16)
             for m, x in p.items()} for p in before]
    same([parts], want)
    for bad in (dict(keep=[3, 4], cu=[0, 3, 3]), dict(keep=[3, 4], cu=[1, 0, 0]),
                dict(keep=[-1, 32], cu=[0, 1, 2]), dict(keep=[0, 0], cu=[0, 2, 2]),
                dict(keep=[20], cu=[0, 1, 1], table=((0, 6), (2, 3))),
                dict(keep=[20], cu=[0, 1, 1], table=((0, -1), (2, 3))),
                dict(keep=[20], cu=[0, 1, 1], out=((9,), (4,))),
                dict(keep=[20, 21], cu=[0, 2, 2], out=((4,), (5,)), start=[-2, 0]),
                dict(keep=[20], cu=[0, 1, 1], out=((4,), (5,)), start=[16, 0])):
        call(**bad)
        reported()
        same([parts], want)


def test_layers_have_to_agree():
    a, _ = pool("e4m3", 4, 2, 16, 0)
    for b in (pool("bf16", 4, 2, 16, 0)[0], pool("e4m3", 5, 2, 16, 0)[0], pool("e4m3", 4, 1, 16, 0)[0],
              pool("e4m3", 4, 2, 32, 0)[0], pool("e4m3", 4, 2, 16, 0, together=True)[0]):
        with pytest.raises(ValueError):
            bs.PagedLayers([a, b])


# -------------------------------------------------- streams and captured graphs --
def test_calls_on_another_stream_and_in_a_graph():
    refs, table, old, new = batch(4, 30, 16, 200, 900, 0.4, 40)
    want = plain.reserve(refs, table, old, new, 16)
    saved = (i32(refs), i32(table))
    R, T, a, b = saved[0].clone(), saved[1].clone(), i32(old), i32(new)
    kv, parts = pools("e4m3", 3, 900, 2, 16, 8)
    before = host(parts)
    out = tuple(torch.empty(30, dtype=torch.int32, device=DEV) for _ in range(3))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bs.attn_skip_pages_reserve(R, T, a, b, 16, out=out, stream=side)
    bs.attn_skip_kv_copy_pages(kv, out[1], out[2], stream=side)
    side.synchronize()
    assert R.tolist() == want[0] and T.tolist() == want[1]
    copied = [{m: plain.copy_pages(x, want[3], want[4]) for m, x in p.items()} for p in before]
    same(parts, copied)
    # The same captured, with the step back; replayed from the start.
    graph = torch.cuda.CUDAGraph()
    R.copy_(saved[0]), T.copy_(saved[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        bs.attn_skip_pages_reserve(R, T, a, b, 16, out=out)
        bs.attn_skip_kv_copy_pages(kv, out[1], out[2])
        bs.attn_skip_pages_fork(R, T, out[0], a, 16)
    for _ in range(2):
        R.copy_(saved[0]), T.copy_(saved[1])
        graph.replay()
        torch.cuda.synchronize()
        back = plain.fork(want[0], want[1], want[2], old, 16)
        assert R.tolist() == back[0] and T.tolist() == want[1]
        same(parts, copied)
    no_error()


@pytest.mark.parametrize("n,max_kv", [(1, 3000), (40, 60)])  # rings and a cluster; a CTA each
def test_compact_on_another_stream_and_in_a_graph(n, max_kv):
    n_pages, table, _, keep, cu, start = rows(8, n, 16, max_kv, True)
    kv, parts = pools("e4m3", 2, n_pages, 2, 16, 4)
    before = host(parts)
    saved = [{m: x.clone() for m, x in p.items()} for p in parts]
    args = i32(keep), i32(cu), i32(table)
    st = i32(start)
    want = [{m: plain.compact(x, keep, cu, table, 16, start) for m, x in p.items()} for p in before]

    def back():
        for p, b in zip(parts, saved):
            for m, x in p.items():
                x.copy_(b[m])
        torch.cuda.synchronize()

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bs.attn_skip_kv_compact(kv, *args, start=st, stream=side)
    side.synchronize()
    same(parts, want)
    back()
    # The table given twice is in place too.
    bs.attn_skip_kv_compact(kv, *args, start=st, out_table=args[2])
    same(parts, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.attn_skip_kv_compact(kv, *args, start=st)
    for _ in range(2):
        back()
        graph.replay()
        torch.cuda.synchronize()
        same(parts, want)
    no_error()


def test_fork_and_reserve_on_another_stream():
    refs, table, old, new = batch(7, 20, 16, 200, 700, 0.3, 40)
    parent = [19 - d for d in range(20)]
    cut = [old[p] // 2 for p in parent]
    want = plain.fork(refs, table, old, cut, 16, parent, [[-1] * len(table[0])] * 20)
    R, T = i32(refs), i32(table)
    side = torch.cuda.Stream()
    a, b, p = i32(old), i32(cut), i32(parent)
    torch.cuda.synchronize()
    out = bs.attn_skip_pages_fork(R, T, a, b, 16, parent=p, stream=side)
    grown = i32([c + 5 for c in cut])
    torch.cuda.synchronize()
    got = bs.attn_skip_pages_reserve(R, out, b, grown, 16, stream=side)
    side.synchronize()
    want = plain.reserve(want[0], want[1], cut, [c + 5 for c in cut], 16)
    assert R.tolist() == want[0] and out.tolist() == want[1]
    assert [x.tolist() for x in got] == list(want[2:5])
    no_error()


# ------------------------------------------------------------------ large pools --
def test_offsets_beyond_32_bits():
    """k and v of 5 GB each: pages whose first byte lies behind 2^32."""
    n_pages, Hkv, ps = 20000, 8, 128
    shape = (n_pages, Hkv, ps, 128)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    high = [n_pages - 1 - i for i in range(6)]
    g = torch.Generator(device=DEV).manual_seed(1)
    for x in (k, v):
        for p in high + [0, 1, 2]:
            x[p] = torch.randn(shape[1:], device=DEV, generator=g).to(torch.bfloat16)
    kv = bs.PagedKV("bf16", k, v)
    before = [[x[p].clone() for p in high] for x in (k, v)]
    bs.attn_skip_kv_copy_pages(kv, i32([high[0], high[1]]), i32([1, high[2]]))
    for x, b in zip((k, v), before):
        assert torch.equal(x[1], b[0]) and torch.equal(x[high[2]], b[1])
    # Rows of two pages move up by 100; the same into other pages.
    table, n = [[high[3], high[4]]], 2 * ps - 100
    bs.attn_skip_kv_compact(kv, i32(range(100, 2 * ps)), i32([0, n]), i32(table),
                            out_table=i32([[high[5], 0]]))
    bs.attn_skip_kv_compact(kv, i32(range(100, 2 * ps)), i32([0, n]), i32(table))
    for x, b in zip((k, v), before):
        rows = torch.cat((b[3], b[4]), 1)  # [Hkv, 2 ps, 128]
        want = torch.cat((rows[:, 100:], rows[:, 2 * ps - 100:]), 1)
        assert torch.equal(torch.cat((x[high[3]], x[high[4]]), 1), want)
        assert torch.equal(x[high[5]], want[:, :ps])
        assert torch.equal(x[0][:, :n - ps], want[:, ps:n])
    no_error()


def test_long_sequences_use_a_few_pages_of_a_wide_table():
    # 2^30 positions in the table, of which three pages are used.
    width = (1 << 30) // 256
    T = torch.full((2, width), -1, dtype=torch.int32, device=DEV)
    T[1, -2:] = i32([5, 7])
    R = i32([0, 0, 0, 0, 0, 1, 0, 1])
    top = (1 << 30) - 300
    # (A length that the pages do not cover would do for the arithmetic: only its end is used.)
    got, src, dst = bs.attn_skip_pages_reserve(R, T, i32([0, top]), i32([256, 1 << 30]), 256)
    assert got.tolist() == [256, 1 << 30] and T[0, 0] == 0 and T[1, -1] == 1 and T[1, -2] == 5
    assert src.tolist() == dst.tolist() == [-1, -1] and R.tolist() == [1, 1, 0, 0, 0, 1, 0, 1]
    no_error()
