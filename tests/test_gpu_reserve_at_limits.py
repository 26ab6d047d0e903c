"""attn_skip_pages_reserve where calls of very different sizes meet: host threads of one
program that reserve at the same time, and the largest batch over the largest pool."""
import random
import threading

import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_threads_that_reserve_for_batches_of_different_sizes():
    """The kernel's limit of shared memory is one for the whole program; the four batches need
    between 50 and 210 KB of it, each thread has counts, tables and a stream of its own."""
    lib, calls, failed = bs.load(), 3000, []
    sizes = ((8192, 1 << 20), (900, 9000), (8192, 9000), (1500, 70000))
    states = []
    for n, n_pages in sizes:
        x = dict(refs=torch.ones(n_pages, dtype=torch.int32, device=DEV),
                 table=torch.full((n, 1), -1, dtype=torch.int32, device=DEV),
                 kv_len=torch.zeros(n, dtype=torch.int32, device=DEV),
                 new_len=torch.ones(n, dtype=torch.int32, device=DEV),
                 stream=torch.cuda.Stream())
        x["out"] = [torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(3)]
        x["refs"][3], x["new_len"][1:] = 0, 0  # one page free, one sequence that asks for it
        x["back"] = x["refs"].clone()
        states.append(x)
    torch.cuda.synchronize()
    gate = threading.Barrier(len(states))

    def work(x):
        args = (x["refs"].data_ptr(), x["refs"].numel(), x["table"].data_ptr(), x["table"].shape[0], 1,
                16, x["kv_len"].data_ptr(), x["new_len"].data_ptr(),
                *(o.data_ptr() for o in x["out"]), x["stream"].cuda_stream)
        gate.wait()
        for _ in range(calls):
            st = lib.attn_skip_pages_reserve(*args)
            if st:
                failed.append((args[3], st))
        with torch.cuda.stream(x["stream"]):
            x["refs"].copy_(x["back"])
        st = lib.attn_skip_pages_reserve(*args)
        if st:
            failed.append((args[3], st))
        x["stream"].synchronize()

    threads = [threading.Thread(target=work, args=(x,)) for x in states]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:5]
    for x in states:
        assert int(x["table"][0, 0]) == 3 and int(x["out"][0][0]) == 1
        assert int(x["refs"].sum()) == x["refs"].numel()
    bs.attn_skip_last_device_error()


def test_the_most_sequences_over_the_largest_pool():
    """8192 sequences of a pool of 2^20 pages (the most shared memory that a call takes): free
    pages far apart, forks that need a copy, sequences that need nothing."""
    r, n, n_pages, ps = random.Random(2), 8192, 1 << 20, 16
    refs = [1] * n_pages
    for p in r.sample(range(n_pages), 7000):
        refs[p] = 0
    held = [p for p in range(n_pages) if refs[p]][:n]
    table, old, new = [], [], []
    for s in range(n):
        a = r.choice((0, 5, 16))
        table.append([held[s], -1, -1])
        if s and r.random() < 0.3:  # a fork of the one before
            a, table[s] = old[s - 1], list(table[s - 1])
            refs[table[s][0]] += 1 if a else 0
        old.append(a)
        new.append(a + r.choice((0, 1, 12, 20)))
    want = plain.reserve(refs, table, old, new, ps)
    R, T = i32(refs), i32(table)
    got = bs.attn_skip_pages_reserve(R, T, i32(old), i32(new), ps)
    assert R.tolist() == want[0] and T.tolist() == want[1]
    assert [x.tolist() for x in got] == list(want[2:5])
    assert sum(x >= 0 for x in want[3]) > 500 and any(a != b for a, b in zip(want[2], new))
    bs.attn_skip_last_device_error()


def test_requests_of_more_than_two_to_the_31_pages():
    """Ten sequences that ask for 2^28 pages each: none fits, and only those that ask for nothing
    go on, before and behind the place where the requests' sum passes 32 bits."""
    n, width = 13, 1 << 28
    T = torch.empty((n, width), dtype=torch.int32, device=DEV)
    T[:, :2] = -1
    R = i32([0, 1, 0, 1, 0])
    old, new = [0] * n, [width] * n
    for s, page in ((1, 1), (12, 3)):  # these grow within their page
        old[s], new[s] = 1, 2
        T[s, 0] = page
    old[11], new[11] = 4, 4  # and this one not at all
    got, src, dst = bs.attn_skip_pages_reserve(R, T, i32(old), i32([4 * x if x == width else x for x in new]),
                                               4)
    assert got.tolist() == [new[s] if s in (1, 11, 12) else 0 for s in range(n)]
    assert src.tolist() == dst.tolist() == [-1] * n and R.tolist() == [0, 1, 0, 1, 0]
    assert T[:, :2].tolist() == [[{1: 1, 12: 3}.get(s, -1), -1] for s in range(n)]
    bs.attn_skip_last_device_error()


@pytest.mark.parametrize("n,n_pages,copies", [
    (2, 4, 1), (3000, 9000, 2999),     # all but the last holder
    (500, 600, 399), (500, 200, 132),  # as far as the free pages go: three for every two sequences
])
def test_copies_of_one_shared_page(n, n_pages, copies):
    """Samples of one prompt of 20 positions, pages of 16; every other one grows into a new page."""
    R = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    R[1] = R[n_pages - 1] = n
    T = i32([[n_pages - 1, 1, -1]] * n)
    new = [21 + 15 * (s % 2) for s in range(n)]
    got, src, dst = bs.attn_skip_pages_reserve(R, T, i32([20] * n), i32(new), 16)
    assert src.tolist() == [1] * copies + [-1] * (n - copies)
    taken = [p for p in range(n_pages - 1) if p != 1]
    # Sequence s copies to its first page; an odd one then takes another.
    first = [3 * (s // 2) + s % 2 for s in range(copies)]
    assert dst.tolist() == [taken[i] for i in first] + [-1] * (n - copies)
    assert R[1] == n - copies and R[n_pages - 1] == n
    served = n if copies == n - 1 else copies
    assert got.tolist() == new[:served] + [20] * (n - served)
    assert T[:copies, 1].tolist() == [taken[i] for i in first]
    assert (T[copies:, 1] == 1).all()
    bs.attn_skip_last_device_error()
