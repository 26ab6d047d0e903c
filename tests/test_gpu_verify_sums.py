"""attn_skip_verify_drafts at rows whose weights sum to 16 and more (scores that nobody has
normalised): a token is written for each, the last one, and rows just below are drawn from."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import DEV, i32, no_error, reported

pytestmark = pytest.mark.gpu


def call(target, n, drafted=(), draft=None, ua=None, us=0.5):
    """Tokens and counts, into arrays that hold something else before."""
    n_seq, total = len(n), sum(n)
    out = (torch.full((n_seq, max(n) + 1), 77777, dtype=torch.int32, device=DEV),
           torch.full((n_seq,), 77777, dtype=torch.int32, device=DEV))
    bs.attn_skip_verify_drafts(target, i32(list(drafted)), i32(np.concatenate(([0], np.cumsum(n)))), max(n),
                               torch.full((total,), 0.75, device=DEV) if ua is None else ua,
                               torch.full((n_seq,), us, device=DEV), draft=draft, out=out)
    return out[0].tolist(), out[1].tolist()


def exact(w, u):
    """The draw of whole units, their sum as it is."""
    w = [int(x) for x in w]
    total, upto = sum(w), 0
    if total == 0 or total >= 1 << 64:
        return len(w) - 1
    num, den = float(np.float32(u)).as_integer_ratio()
    for t, x in enumerate(w):
        upto += x
        if upto > num * total // den:
            return t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [17, 40, 700, 2049, 50001, 128000])
@pytest.mark.parametrize("x", [1.9375, 1.0, 0.5])
def test_constant_rows(V, x, dtype):
    """Among them sums that are multiples of 16, whose 64 bits are zero."""
    for n_seq in (1, 3, 300):
        p = torch.zeros(n_seq, V, device=DEV, dtype=dtype)
        p[:, 3] = 0.25
        p[0, :-1] = x
        p[n_seq // 2, :min(V - 1, int(16 / x) * (V // int(16 / x)))] = x
        tokens, accepted = call(p, [0] * n_seq)
        assert accepted == [0] * n_seq
        for s in {0, n_seq // 2, n_seq - 1}:
            assert tokens[s] == [exact(plain.units(p[s].double().cpu().numpy()), 0.5)]
        assert V * x < 17 or tokens[0] == [V - 1]
    no_error()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3000, 60001])
@pytest.mark.parametrize("together", [True, False])
def test_sums_about_sixteen(V, together, dtype):
    """Large values next to one another or all over the row, up to 16 less a little, 16, and on."""
    for last in (0.5 - 2.0 ** -8, 0.5, 0.5 + 2.0 ** -8, 16.5):
        p = torch.zeros(2, V, device=DEV, dtype=dtype)
        at = torch.arange(31) + 100 if together else torch.arange(31) * (V // 33) + 5
        p[0, at] = 0.5
        at = torch.arange(min(33, max(1, int(2 * last)))) + V - 40
        p[0, at] = last / len(at)
        p[1, 9] = 1.0
        w = plain.units(p[0].double().cpu().numpy())
        assert (sum(int(x) for x in w) >= 1 << 64) == (last >= 0.5)
        for u in (0.0, 0.4, 1 - 2.0 ** -24):
            tokens, _ = call(p, [0, 0], us=u)
            assert tokens == [[exact(w, u)], [9]]
            assert last < 0.5 or tokens[0] == [V - 1]
    no_error()


@pytest.mark.parametrize("V", [1000, 40000])
def test_differences_and_look_ups(V):
    """What counts is the sum of the weights that are drawn from."""
    p = torch.zeros(2, V, device=DEV)
    p[0, :200] = 1.5
    q = torch.zeros(1, V, device=DEV)
    q[0, :200] = 1.4375  # p - q sums to 12.5, p to 300
    q[0, 300] = 1.0      # the drafted token, which has p = 0
    w = np.maximum(plain.units(p[0].double().cpu().numpy()) - plain.units(q[0].double().cpu().numpy()), 0)
    assert call(p, [1], [300], q) == ([[exact(w, 0.5), -1]], [0]) and exact(w, 0.5) == 100
    q[0, :200] = 1.375   # p - q sums to 25
    assert call(p, [1], [300], q) == ([[V - 1, -1]], [0])
    q[0, :200] = 1.34    # and to about 32
    assert call(p, [1], [300], q) == ([[V - 1, -1]], [0])
    p[0, :200], q[0, :200] = 1.25, 1.0 - 2.0 ** -2
    p[0, 64:200] = 0.75  # to 32 exactly: no empty difference
    assert call(p, [1], [300], q) == ([[V - 1, -1]], [0])
    # A look-up: all but the token itself.
    p.zero_()
    p[0, 10:25], p[0, 700] = 1.0, 0.75
    assert call(p, [1], [700]) == ([[17, -1]], [0])
    p[0, 26] = 1.0
    assert call(p, [1], [700]) == ([[V - 1, -1]], [0])
    no_error()


def test_values_that_count_as_zero_among_too_many():
    p = torch.full((1, 5000), 1.0, device=DEV)
    p[0, 4000], p[0, 17] = float("nan"), -1.0
    assert call(p, [0])[0] == [[4999]]
    reported()
    p[0, 16:] = 0.0  # sixteen ones before
    p[0, 20] = float("nan")
    assert call(p, [0])[0] == [[4999]]
    reported()
    p[0, 0] = 0.5
    assert call(p, [0], us=0.0)[0] == [[0]]
    reported()


def test_many_values_halfway_between_steps():
    """2^26 tokens of 2^-22 sum to 16; without one of them they are drawn from."""
    V = 1 << 26
    p = torch.full((1, V), 2.0 ** -22, device=DEV)
    assert call(p, [0]) == ([[V - 1]], [0])
    assert call(p, [0], us=0.0) == ([[V - 1]], [0])
    p[0, V - 5] = 0.0
    for u in (0.0, 0.25, 0.75):
        assert call(p, [0], us=u) == ([[int(u * (V - 1))]], [0])
    p = p.to(torch.bfloat16)
    assert call(p, [0], us=0.25) == ([[int(0.25 * (V - 1))]], [0])
    p[0, V - 5] = 2.0 ** -22
    assert call(p, [0], us=0.25) == ([[V - 1]], [0])
    no_error()
