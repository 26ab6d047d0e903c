"""Refusals of the calls around the paged cache that go with how their arrays lie to one
another (on the host: no call here reaches a launch)."""
import pytest

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_pages_host import A, lib, reserve  # noqa: F401 (lib: the fixture)


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
