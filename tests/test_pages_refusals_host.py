"""Refusals of the calls around the paged cache that go with how their arrays lie to one
another (on the host: no call here reaches a launch)."""
import pytest

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_paged_host import append, chunk, gather, pages
from tests.test_pages_host import A, compact, copy, layers, lib, reserve  # noqa: F401 (lib: the fixture)


@pytest.mark.parametrize("lengths", ["kv_len", "new_len"])
@pytest.mark.parametrize("copies", ["src", "dst"])
def test_reserve_rejects_one_array_for_lengths_and_pages_to_copy(lib, lengths, copies):  # noqa: F811
    """A copy's page is written while other lengths are still to be read."""
    at = dict(kv_len=5 * A, new_len=6 * A)
    assert reserve(lib, **at, **{copies: at[lengths]}) == bs.ATTN_EINVAL
    # (Apart the call gets past its arrays: refused for its size.)
    assert reserve(lib, **at, n_seq=8193) == bs.ATTN_EUNSUPPORTED
    # The lengths that are granted may take the place of the old ones, or of the new ones.
    for got in at.values():
        assert reserve(lib, **at, got=got, n_seq=8193) == bs.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("again", [dict(), dict(v=4 * A), dict(k=4 * A)])
def test_compact_rejects_a_cache_that_stands_there_twice(lib, again):  # noqa: F811
    """Its rows would move twice in place.  (n_seq is refused behind it.)"""
    one, other = pages(k=2 * A, v=3 * A), pages(k=5 * A, v=6 * A)
    twice = pages(**dict(dict(k=2 * A, v=3 * A), **again))
    assert compact(lib, kv=layers(one, other, twice), n=3) == bs.ATTN_EINVAL
    assert compact(lib, kv=layers(other, one, twice), n=3) == bs.ATTN_EINVAL
    assert compact(lib, kv=layers(other, twice, one), n=3) == bs.ATTN_EINVAL
    many = dict(n_seq=1 << 30)
    assert compact(lib, kv=layers(other, one), n=2, **many) == bs.ATTN_EUNSUPPORTED
    assert compact(lib, kv=layers(one, other), n=2, **many) == bs.ATTN_EUNSUPPORTED
    assert compact(lib, kv=layers(one, other, twice), n=3, out=A) == bs.ATTN_EINVAL  # (its table)
    # Rows that go to other pages, and whole pages, may go twice.
    assert compact(lib, kv=layers(one, other, twice), n=3, out=2 * A, out_pages=4,
                   **many) == bs.ATTN_EUNSUPPORTED
    assert copy(lib, kv=layers(one, other, twice), n=3, pairs=0) == bs.ATTN_OK


@pytest.mark.parametrize("number", [(1 << 30) + 1, (1 << 31) - 1])
def test_numbers_beyond_int_loops(lib, number):  # noqa: F811
    """A block's threads step through pairs and sequences by its size: beyond 2^31 less that much
    the step would wrap."""
    one = dict(kv=layers(pages(Hkv=1)))
    assert copy(lib, **one, pairs=number) == bs.ATTN_EUNSUPPORTED
    assert compact(lib, **one, n_seq=number) == bs.ATTN_EUNSUPPORTED
    for call in (append, gather, chunk):
        assert call(lib, n_seq=number, total=0) == bs.ATTN_EUNSUPPORTED
