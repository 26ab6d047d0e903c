"""attn_skip_pages_fork reports every page id out of range that it meets: in entries that are
handed on, whether or not their counts change, and in those that are let go."""
import pytest

from block_sparse_attention_online_gb300 import binding as bs
from tests.test_gpu_pages import i32, no_error, reported

pytestmark = pytest.mark.gpu
PS = 4


def call(table, old, new, parent, n_pages):
    R = i32([1] * n_pages)
    out = bs.attn_skip_pages_fork(R, i32(table), i32(old), i32(new), PS,
                                  parent=None if parent is None else i32(parent))
    return R.tolist(), out.tolist()


@pytest.mark.parametrize("bad", [-1, 9, 1 << 30, -(1 << 31)])
@pytest.mark.parametrize("followers", [1, 2, 3, 40])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_ids_that_are_handed_on(bad, followers, at):
    row = [3, 4, 5]
    row[at] = bad
    refs, out = call([row, [6, 7, 8]], [12, 12], [12] * (followers + 1), [0] * followers + [1], 9)
    reported()
    assert out == [row] * followers + [[6, 7, 8]]
    assert refs == [followers if p in row else 1 for p in range(9)]


@pytest.mark.parametrize("n", [1, 255, 256, 257, 2048, 2049, 5000])
def test_one_among_many_entries(n):
    """By every place that a thread takes, one follower: no count changes."""
    for at in sorted({0, n // 2, n - 1}):
        row = list(range(n))
        row[at] = n
        refs, out = call([row], [n * PS], [n * PS], [0], n)
        reported()
        assert out == [row] and refs == [1] * n
    refs, out = call([list(range(n))], [n * PS], [n * PS], [0], n)
    no_error()
    assert refs == [1] * n


def test_ids_that_are_let_go_or_never_used():
    # Behind the cached length: not looked at, whoever follows.
    assert call([[0, 99, -7]], [4], [4], [0], 3)[0] == [1, 1, 1]
    no_error()
    # Cut off, with a follower, without one, and in place.
    for new, parent in ([4], [0]), ([0], [-1]), ([4], None):
        refs, _ = call([[0, 99, 1]], [12], new, parent, 3)
        reported()
        assert refs == [0 if new == [0] else 1, 0, 1]
    # Kept in place: nothing of it is read.
    assert call([[0, 99, 1]], [12], [12], None, 3)[0] == [1, 1, 1]
    no_error()
