"""Refusals of the page bookkeeping, of the calls that move pages and rows and of the
check of drafted tokens (on the host: no call here reaches a launch), and properties of
their plain implementations (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from block_sparse_attention_online_gb300 import build as B
from tests import pages_plain as plain
from tests.test_paged_host import BAD_PAGES, UNSUPPORTED_PAGES, pages

A = 0x10000  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return bs.load()


def layers(*kv):
    return ctypes.byref((bs._KvPages * len(kv))(*kv))


def reserve(lib, **kw):
    a = dict(refs=A, n_pages=9, table=A, n_seq=2, max_pages=4, ps=16, kv_len=A, new_len=A, got=A,
             src=2 * A, dst=3 * A, stream=None)
    a.update(kw)
    return lib.attn_skip_pages_reserve(*a.values())


def fork(lib, **kw):
    a = dict(refs=A, n_pages=9, table=A, n_seq=2, max_pages=4, ps=16, kv_len=A, new_len=A, n_new=3,
             parent=A, out=2 * A, stream=None)
    a.update(kw)
    return lib.attn_skip_pages_fork(*a.values())


def copy(lib, one=None, **kw):
    a = dict(kv=layers(one or pages()), n=1, pairs=3, src=A, dst=A, stream=None)
    a.update(kw)
    return lib.attn_skip_kv_copy_pages(*a.values())


def compact(lib, one=None, **kw):
    a = dict(kv=layers(one or pages()), n=1, n_seq=2, total=5, cu=A, keep=A, per_head=0, start=A,
             table=A, max_pages=4, out=None, out_pages=0, stream=None)
    a.update(kw)
    return lib.attn_skip_kv_compact(*a.values())


def verify(lib, **kw):
    a = dict(target=A, ts=100, draft=A, ds=100, dt=1, V=100, n_seq=2, total=3, max_draft=2,
             drafted=A, cu=A, ua=A, us=A, tokens=A, acc=2 * A, stream=None)
    a.update(kw)
    return lib.attn_skip_verify_drafts(*a.values())


TABLES = [dict(refs=None), dict(refs=A + 2), dict(n_pages=0), dict(table=None), dict(table=A + 1),
          dict(n_seq=0), dict(max_pages=0), dict(ps=0), dict(kv_len=None), dict(kv_len=A + 2),
          dict(new_len=None), dict(new_len=A + 1)]


@pytest.mark.parametrize("kw", TABLES + [dict(got=None), dict(src=None), dict(dst=A + 2),
                                         dict(got=2 * A), dict(src=3 * A), dict(dst=A)])
def test_reserve_rejects_invalid_arguments(lib, kw):
    assert reserve(lib, **kw) == bs.ATTN_EINVAL


@pytest.mark.parametrize("kw", [dict(n_seq=8193), dict(n_pages=(1 << 20) + 1),
                                dict(max_pages=1 << 28), dict(ps=1 << 30, max_pages=2)])
def test_reserve_limits(lib, kw):
    assert reserve(lib, **kw) == bs.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("kw", TABLES + [dict(n_new=0), dict(out=None), dict(out=A), dict(parent=A + 2),
                                         dict(out=2 * A + 2)])
def test_fork_rejects_invalid_arguments(lib, kw):
    assert fork(lib, **kw) == bs.ATTN_EINVAL


@pytest.mark.parametrize("kw", [dict(n_seq=65537), dict(n_new=65537), dict(max_pages=1 << 28)])
def test_fork_limits(lib, kw):
    assert fork(lib, **kw) == bs.ATTN_EUNSUPPORTED


def test_fork_without_parents_needs_no_second_table(lib):
    # (Refused for another reason: the call has got past the tables.)
    assert fork(lib, parent=None, out=None, n_new=0, n_seq=65537) == bs.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("call", [copy, compact])
def test_layers_are_checked(lib, call):
    for kw in BAD_PAGES:
        assert call(lib, pages(**kw)) == bs.ATTN_EINVAL, kw
        assert call(lib, kv=layers(pages(), pages(**kw)), n=2) == bs.ATTN_EINVAL
    for kw in UNSUPPORTED_PAGES:
        assert call(lib, pages(**kw)) == bs.ATTN_EUNSUPPORTED, kw
    for kw in (dict(format=0), dict(n_pages=9), dict(page_size=32), dict(Hkv=1),
               dict(page_stride=1 << 20)):  # layers that differ
        assert call(lib, kv=layers(pages(), pages(**kw)), n=2) == bs.ATTN_EINVAL, kw
    assert call(lib, n=0) == bs.ATTN_EINVAL
    assert call(lib, kv=None) == bs.ATTN_EINVAL


@pytest.mark.parametrize("kw", [dict(pairs=-1), dict(src=None), dict(dst=None), dict(src=A + 2)])
def test_copy_pages_rejects_invalid_arguments(lib, kw):
    assert copy(lib, **kw) == bs.ATTN_EINVAL


def test_copy_pages_and_compact_limits(lib):
    assert copy(lib, pages(page_size=128, Hkv=(1 << 17) + 1)) == bs.ATTN_EUNSUPPORTED
    assert copy(lib, pages(page_size=128, Hkv=1 << 17), pairs=0) == bs.ATTN_OK
    assert compact(lib, pages(Hkv=1 << 10), n_seq=1 << 21) == bs.ATTN_EUNSUPPORTED
    assert compact(lib, total=(1 << 30) + 1) == bs.ATTN_EUNSUPPORTED


def test_nothing_to_do(lib):
    assert copy(lib, pairs=0, src=None, dst=None) == bs.ATTN_OK
    assert compact(lib, total=0, keep=None) == bs.ATTN_OK


@pytest.mark.parametrize("kw", [
    dict(n_seq=0), dict(total=-1), dict(cu=None), dict(cu=A + 2), dict(keep=None), dict(keep=A + 1),
    dict(start=A + 2), dict(table=None), dict(max_pages=0), dict(out=2 * A, out_pages=0),
    dict(out=2 * A + 1, out_pages=4),
])
def test_compact_rejects_invalid_arguments(lib, kw):
    assert compact(lib, **kw) == bs.ATTN_EINVAL
    assert compact(lib, out=2 * A, out_pages=1 << 28) == bs.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(target=None), dict(target=A + 2), dict(draft=A + 1), dict(ts=99), dict(ds=99), dict(dt=2),
    dict(V=0), dict(n_seq=0), dict(total=-1), dict(max_draft=-1), dict(drafted=None), dict(cu=None),
    dict(ua=None), dict(us=None), dict(tokens=None), dict(acc=None), dict(us=A + 2),
    dict(tokens=A + 1), dict(ts=1 << 40), dict(dt=0, target=A + 1), dict(tokens=2 * A),
])
def test_verify_rejects_invalid_arguments(lib, kw):
    assert verify(lib, **kw) == bs.ATTN_EINVAL


def test_verify_limits(lib):
    assert verify(lib, V=(1 << 28) + 1, ts=1 << 29, ds=1 << 29) == bs.ATTN_EUNSUPPORTED


def test_bindings_refuse_tensors_of_the_cpu():
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        bs.attn_skip_pages_reserve(i, i.view(2, 2), i[:2], i[:2], 16)
    with pytest.raises(ValueError):
        bs.attn_skip_pages_fork(i, i.view(2, 2), i[:2], i[:2], 16)
    with pytest.raises(ValueError):
        bs.attn_skip_verify_drafts(torch.zeros(3, 5), i[:2], i[:2], 2, torch.zeros(2), torch.zeros(1))
    with pytest.raises(ValueError):
        bs.PagedLayers([])


# -------------------------------------------------- the plain implementations --
def test_plain_reserve_by_hand():
    # Pages of 4; page 1 is held by all three sequences, 3 of its 4 rows used.
    refs, table = [0, 3, 0, 1, 0], [[3, 1, -1], [1, -1, -1], [1, -1, -1]]
    got = plain.reserve(refs, table, [7, 3, 3], [8, 5, 4], 4)
    # The first copies (page 0), the second copies (2) and goes on (4), the last writes in place.
    assert got == ([1, 1, 1, 1, 1], [[3, 0, -1], [2, 4, -1], [1, -1, -1]], [8, 5, 4], [1, 1, -1],
                   [0, 2, -1], False)
    # Two free pages: the second does not fit, nor does the third, which would write into
    # the page that the second still holds.
    refs = [0, 3, 0, 1, 1]
    got = plain.reserve(refs, table, [7, 3, 3], [8, 5, 4], 4)
    assert got[2:] == ([8, 3, 3], [1, -1, -1], [0, -1, -1], False)
    assert got[0] == [1, 2, 0, 1, 1]


def test_plain_fork_by_hand():
    refs, table = [1, 1, 1, 0], [[0, 1], [2, -1]]
    got = plain.fork(refs, table, [7, 2], [7, 5, 3, 0], 4, [0, 0, 0, -1], [[9, 9]] * 4)
    assert got == ([3, 2, 0, 0], [[0, 1], [0, 1], [0, 9], [9, 9]])
    assert plain.fork(refs, table, [7, 2], [4, 0], 4) == ([1, 0, 0, 0], table)


def test_plain_verify_draws_from_the_target():
    """Over a grid of random numbers the first token's frequencies are the target's: with g
    steps a frequency is off by at most one step for every boundary it has, V + 1 of them in
    each of the two numbers."""
    r = np.random.default_rng(3)
    V, g = 5, 400
    p, q = r.dirichlet(np.ones(V), 2).astype(np.float32).astype(np.float64), r.dirichlet(np.ones(V))
    q = q.astype(np.float32).astype(np.float64)
    u = (np.arange(g) + 0.5).astype(np.float32) / g
    for draft in (q, None):
        count = np.zeros(V)
        for x in range(V):
            weight = q[x] if draft is not None else float(x == 2)
            if not weight:
                continue
            for ua in u[::20]:
                for us in u[::20]:
                    t, _ = plain.verify(p, [x], [0, 1], 1, [ua], [us],
                                        None if draft is None else q[None])
                    count[t[0, 0]] += weight / 400
        assert np.abs(count / count.sum() - p[0]).max() < 2 * (V + 1) / 20


def test_plain_draw_takes_whole_units():
    assert plain.units([0.5, 2.0 ** -60, 2.0 ** -61, 2.0, np.nan, -1.0, 1.5]).tolist() == [
        1 << 59, 1, 0, 0, 0, 0, 3 << 59]
    w = plain.units([0.0, 0.25, 0.0, 0.25])
    assert [plain.draw(w, u) for u in (0.0, 0.49, 0.5, 0.99)] == [1, 1, 3, 3]
    assert plain.draw(plain.units([0.0, 0.0]), 0.3) == 1
