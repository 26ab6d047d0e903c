"""attn_skip_verify_drafts against the plain implementation in whole numbers: the same
tokens everywhere (sums of whole units are exact in any order, acceptance compares a
product that 64 bits hold exactly)."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import DEV, i32, no_error, reported

pytestmark = pytest.mark.gpu


def inputs(seed, n, V, dtype=torch.float32, probs=True, sharp=3.0, noise=0.7, cut=False, pad=(0, 0)):
    """Sequences with n[s] drafted tokens; ``pad``: spare columns and a start inside a row,
    so that rows are not aligned."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    total, rows = sum(n), sum(n) + len(n)

    def dist(z):
        p = torch.softmax(z, -1)
        if cut:
            p = torch.where(p < p.amax(-1, keepdim=True) / 50, torch.zeros_like(p), p)
            p = p / p.sum(-1, keepdim=True)
        return p

    def stored(p):
        wide = torch.full((p.shape[0], V + pad[0]), 9.0, device=DEV).to(dtype)
        wide[:, pad[1]:pad[1] + V] = p.to(dtype)
        return wide[:, pad[1]:pad[1] + V]

    z = sharp * torch.randn(rows, V, device=DEV, generator=g)
    last = np.cumsum(np.asarray(n) + 1) - 1
    inner = torch.tensor(np.setdiff1d(np.arange(rows), last), device=DEV, dtype=torch.long)
    q = dist(z[inner] + noise * torch.randn(total, V, device=DEV, generator=g))
    if total:
        e = torch.empty_like(q).exponential_(generator=g)
        x = ((q / e) if probs else q).argmax(-1).to(torch.int32)
    else:
        x = i32([])
    return dict(target=stored(dist(z)), drafted=x, cu=i32(np.concatenate(([0], np.cumsum(n)))),
                max_draft=max(n), u_accept=torch.rand(total, device=DEV, generator=g),
                u_sample=torch.rand(len(n), device=DEV, generator=g),
                draft=stored(q) if probs else None)


def call(a, **kw):
    return bs.attn_skip_verify_drafts(a["target"], a["drafted"], a["cu"], a["max_draft"],
                                      a["u_accept"], a["u_sample"], draft=a["draft"], **kw)


def want(a):
    h = {k: v.double().cpu().numpy() if torch.is_tensor(v) else v for k, v in a.items()}
    return plain.verify(h["target"], h["drafted"].astype(int), h["cu"].astype(int), h["max_draft"],
                        h["u_accept"], h["u_sample"], h["draft"])


def check(a):
    tokens, accepted = call(a)
    t, n = want(a)
    assert np.array_equal(accepted.cpu().numpy(), n)
    assert np.array_equal(tokens.cpu().numpy(), t)
    return t, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("V,n,pad", [
    (1, [1, 0], (0, 0)), (2, [3, 0, 1], (0, 0)), (31, [4, 2], (3, 1)), (32, [1], (0, 0)),
    (33, [5, 0, 5, 1], (0, 0)), (127, [2, 2, 2], (7, 5)), (128, [0, 0], (0, 0)),
    (2049, [7, 3, 0, 16], (1, 1)), (4096, [4, 4], (0, 0)), (32000, [4], (0, 0)),
    (50001, [3, 0, 7, 5, 1], (0, 0)), (128000, [5, 2], (3, 2)), (270001, [2], (0, 0)),
])
def test_tokens(V, n, pad, probs, dtype):
    for seed in range(4):
        check(inputs(seed, n, V, dtype, probs, pad=pad, cut=seed == 1, noise=(0.7, 0.1, 2.0, 0.02)[seed]))
    no_error()


@pytest.mark.parametrize("V", [1, 2, 33, 513, 5000, 60001])
def test_rows_that_start_in_either_half_of_a_word(V):
    """bf16 rows at even and odd elements, target and draft alike or not, NaN all round."""
    a = inputs(61, [2, 0, 1, 3], V, torch.bfloat16)
    for spare in (2, 3):
        for at_p in (0, 1):
            for at_q in (0, 1):
                b = dict(a)
                for name, at in (("target", at_p), ("draft", at_q)):
                    wide = torch.full((a[name].shape[0], V + spare), float("nan"), dtype=torch.bfloat16,
                                      device=DEV)
                    wide[:, at:at + V] = a[name]
                    b[name] = wide[:, at:at + V]
                for u in (0.0, 0.5, 1 - 2.0 ** -24):
                    b["u_sample"] = torch.full((4,), u, device=DEV)
                    check(b)
                check(dict(b, draft=None, drafted=torch.clamp(a["drafted"], max=V - 1)))
    no_error()


@pytest.mark.parametrize("V,dtype", [(1300003, torch.float32), (9000001, torch.bfloat16)])
def test_vocabularies_of_millions(V, dtype):
    for seed, probs in ((1, True), (2, False)):
        check(inputs(seed, [1, 0], V, dtype, probs, sharp=1.0))
    no_error()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [3, 257, 1031, 20000])
def test_rows_that_start_anywhere_in_sixteen_bytes(V, dtype):
    """Target and draft as far from a border as each other or not, NaN all round."""
    a = inputs(62, [1, 0, 2], V, dtype)
    each = 16 // a["target"].element_size()
    for at_p in range(each):
        for at_q in range(each):
            b = dict(a)
            for name, at in (("target", at_p), ("draft", at_q)):
                n = a[name].shape[0]
                wide = torch.full((n, (V + 2 * each) // each * each), float("nan"), dtype=dtype, device=DEV)
                wide[:, at:at + V] = a[name]
                b[name] = wide[:, at:at + V]
            check(b)
            b["u_sample"] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.0], device=DEV)
            check(b)
    no_error()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p,q", [(5, 3), (7, 5), (2, 1), (9, 7), (6.5, 0.5)])
@pytest.mark.parametrize("step", [2.0 ** -22, 2.0 ** -44])
def test_constant_rows_halfway_between_steps(p, q, step, dtype):
    """p - q rounds the same way for every token, as far as it can."""
    V = 20011
    for rows in (False, True):
        target = torch.full((2, V), p * step, device=DEV, dtype=dtype)
        draft = torch.full((1, V), q * step, device=DEV, dtype=dtype) if rows else None
        target[0, 4097] = 0.0
        for u in (0.0, 0.25, 0.9, 1 - 2.0 ** -24):
            check(dict(target=target, drafted=i32([4097]), cu=i32([0, 1]), max_draft=1,
                       u_accept=torch.full((1,), 0.5, device=DEV),
                       u_sample=torch.full((1,), u, device=DEV), draft=draft))
    no_error()


def test_rows_that_sum_to_too_much_harm_nothing():
    """(Their token means nothing.)"""
    for V in (40, 3000, 100000):
        a = inputs(1, [1, 0, 0], V, probs=False)
        good = want(a)
        a["target"][2] = 1.9
        tokens, n = call(a)
        assert n.tolist() == good[1].tolist()
        assert np.array_equal(tokens[[0, 2]].cpu().numpy(), good[0][[0, 2]])
    no_error()


def test_many_drafts_and_many_sequences():
    check(inputs(1, [600, 3], 50, noise=0.0))      # more drafts than threads of a CTA
    check(inputs(2, [1] * 700 + [0] * 300, 1000))
    t, n = check(inputs(3, [40, 30], 3000, noise=0.0))
    assert (n == [40, 30]).all()  # q = p: u q < p always
    no_error()


def test_nothing_drafted():
    a = inputs(5, [0, 0, 0], 5000)
    t, n = check(a)
    assert t.shape == (3, 1) and (n == 0).all()
    no_error()


def test_residual_of_zero_everywhere_falls_back_to_the_target():
    # p = 0 at the drafted token and p <= q elsewhere: nothing is left of p - q.
    V = 5000
    p = torch.zeros(2, V, device=DEV)
    p[:, 100:200] = 2.0 ** -8
    q = p[:1].clone()
    q[0, 7] = 0.5
    for u in (0.0, 0.3, 0.9999999):
        a = dict(target=p, draft=q, drafted=i32([7]), cu=i32([0, 1]), max_draft=1,
                 u_accept=torch.zeros(1, device=DEV), u_sample=torch.full((1,), u, device=DEV))
        t, n = check(a)
        assert n[0] == 0 and 100 <= t[0, 0] < 200
    # A look-up whose token holds all of p that there is.
    p = torch.zeros(2, V, device=DEV)
    p[:, 9] = 0.5
    a = dict(target=p, draft=None, drafted=i32([9]), cu=i32([0, 1]), max_draft=1,
             u_accept=torch.full((1,), 0.75, device=DEV), u_sample=torch.full((1,), 0.5, device=DEV))
    t, n = check(a)
    assert n[0] == 0 and t[0, 0] == 9
    no_error()


@pytest.mark.parametrize("V", [1, 40, 9000])
def test_rows_of_zeros_and_borders(V):
    u = torch.tensor([0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24], device=DEV)
    base = dict(draft=None, drafted=i32([]), cu=i32([0] * 5), max_draft=0,
                u_accept=torch.zeros(0, device=DEV), u_sample=u)
    t, _ = check(dict(base, target=torch.zeros(4, V, device=DEV)))
    assert (t == V - 1).all()
    # Thresholds that lie on sums: a sum has to be above.
    p = torch.full((4, V), 2.0 ** -14, device=DEV)
    check(dict(base, target=p))
    # Weights of one unit of 2^-60, and below.
    p = torch.full((4, V), 2.0 ** -61, device=DEV)
    p[:, V // 2] = 2.0 ** -60
    t, _ = check(dict(base, target=p))
    assert (t == V // 2).all()
    no_error()


def test_unnormalised_rows_up_to_sixteen():
    p = torch.rand(3, 8000, device=DEV, generator=torch.Generator(device=DEV).manual_seed(0))
    p = p * (15.9 / p.sum(-1, keepdim=True))
    check(dict(target=p, draft=None, drafted=i32([]), cu=i32([0, 0, 0, 0]), max_draft=0,
               u_accept=torch.zeros(0, device=DEV),
               u_sample=torch.tensor([0.1, 0.5, 0.99], device=DEV)))
    no_error()


def test_values_out_of_range_count_as_zero_and_are_reported():
    a = inputs(8, [0, 0, 0, 0, 0], 3000)
    for i, x in enumerate((float("nan"), -0.25, 2.0, float("inf"))):
        a["target"][i, 5 + i] = x
    a["target"][4, 9] = -0.0
    check(a)
    reported()
    a["target"][:4] = a["target"][4]
    check(a)
    no_error()
    # Random numbers outside [0, 1).
    for u in (1.0, 7.0, -0.5, float("nan")):
        a["u_sample"][1] = u
        tokens, _ = call(a)
        reported()
        b = dict(a, u_sample=a["u_sample"].clone())
        b["u_sample"][1] = 1 - 2.0 ** -24 if u >= 1 else 0.0
        assert np.array_equal(tokens.cpu().numpy(), want(b)[0])
    # Drafted tokens outside [0, V) are rejected.
    for probs in (True, False):
        for x in (-1, 3000, 1 << 30):
            a = inputs(9, [3, 2], 3000, probs=probs, noise=0.0)
            a["drafted"][1] = x
            tokens, n = call(a)
            reported()
            t, m = want(a)
            assert np.array_equal(tokens.cpu().numpy(), t) and n.tolist() == m.tolist()
            assert n[0] <= 1


def test_bad_bounds_and_rows_behind_the_last_sequence():
    a = inputs(11, [3, 2, 4], 700)
    t, n = want(a)
    for s, cu in ((0, [-1, 3, 5, 9]), (2, [0, 3, 5, 10]), (1, [0, 3, 2, 9]), (2, [0, 3, 5, 4]),
                  (0, [0, 5, 5, 9])):
        b = dict(a, cu=i32(cu))
        tokens, acc = call(b)
        reported()
        assert (tokens[s] == -1).all() and acc[s] == -1
    # A padded batch: tokens, numbers and rows behind the last sequence may hold anything.
    b = dict(a, drafted=torch.cat((a["drafted"], i32([1 << 30] * 3))),
             u_accept=torch.cat((a["u_accept"], torch.full((3,), float("nan"), device=DEV))),
             draft=torch.cat((a["draft"], torch.full((3, 700), float("nan"), device=DEV))),
             target=torch.cat((a["target"], torch.full((5, 700), float("nan"), device=DEV))))
    tokens, acc = call(b)
    no_error()
    assert np.array_equal(tokens.cpu().numpy(), t) and np.array_equal(acc.cpu().numpy(), n)


def test_max_draft_is_a_bound():
    a = inputs(14, [3, 0, 1], 5000)
    t, n = want(dict(a, max_draft=9))
    assert t.shape == (3, 10)
    tokens, accepted = call(dict(a, max_draft=9))
    assert np.array_equal(tokens.cpu().numpy(), t) and np.array_equal(accepted.cpu().numpy(), n)
    no_error()
    tokens, accepted = call(dict(a, max_draft=2))  # one sequence has more
    reported()
    assert accepted.tolist() == [-1] + n[1:].tolist() and (tokens[0] == -1).all()
    assert np.array_equal(tokens[1:].cpu().numpy(), t[1:, :3])


def test_refusals():
    a = inputs(1, [2, 1], 60)
    for bad in (dict(target=a["target"].double()), dict(target=a["target"][:4]),
                dict(draft=a["draft"][:2]), dict(draft=a["draft"].bfloat16()),
                dict(draft=a["draft"][:, :50]), dict(u_accept=a["u_accept"][:2]),
                dict(u_sample=a["u_sample"].double()), dict(drafted=a["drafted"].long()),
                dict(cu=a["cu"].cpu()), dict(target=a["target"].t().contiguous().t()),
                dict(target=a["target"][:1].expand(5, 60)), dict(max_draft=-1)):
        with pytest.raises((ValueError, TypeError)):
            call(dict(a, **bad))


def test_given_outputs_another_stream_and_a_graph():
    a = inputs(21, [3, 0, 5], 20001, torch.bfloat16)
    t, n = want(a)
    out = (torch.full((3, 6), 77, dtype=torch.int32, device=DEV),
           torch.full((3,), 77, dtype=torch.int32, device=DEV))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert call(a, out=out, stream=side)[0] is out[0]
    side.synchronize()
    assert np.array_equal(out[0].cpu().numpy(), t) and np.array_equal(out[1].cpu().numpy(), n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, out=out)
    for seed in (22, 23):  # new numbers in the same buffers
        b = inputs(seed, [3, 0, 5], 20001, torch.bfloat16)
        for k in ("target", "drafted", "u_accept", "u_sample", "draft"):
            a[k].copy_(b[k])
        graph.replay()
        torch.cuda.synchronize()
        t, n = want(b)
        assert np.array_equal(out[0].cpu().numpy(), t) and np.array_equal(out[1].cpu().numpy(), n)
    no_error()


def test_rows_far_apart():
    """Rows 2^30 elements apart: the last one starts behind 2^32."""
    V, stride = 5000, 1 << 30
    a = inputs(31, [3, 1], V, torch.bfloat16)
    far = torch.empty(5 * stride + V, dtype=torch.bfloat16, device=DEV)
    target = far.as_strided((6, V), (stride, 1))
    target.copy_(a["target"])
    t, n = want(a)
    tokens, accepted = call(dict(a, target=target))
    assert np.array_equal(tokens.cpu().numpy(), t) and np.array_equal(accepted.cpu().numpy(), n)
    draft = far[7:].as_strided((4, V), (stride, 1))
    draft.copy_(a["draft"])
    tokens, accepted = call(dict(a, draft=draft))
    assert np.array_equal(tokens.cpu().numpy(), t) and np.array_equal(accepted.cpu().numpy(), n)
    no_error()


def test_calls_on_two_streams_at_once():
    cases = [inputs(40 + i, [2, 0, 4, 1], 30000) for i in range(2)]
    wants = [want(a) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[call(a, stream=s) for _ in range(5)] for a, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for runs, (t, n) in zip(got, wants):
        for tokens, accepted in runs:
            assert np.array_equal(tokens.cpu().numpy(), t) and np.array_equal(accepted.cpu().numpy(), n)
    no_error()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_few_long_rows_on_two_streams_and_in_graphs(dtype):
    """Clusters of sixteen side by side, and replayed with other inputs."""
    cases = [inputs(70 + i, [2, 0, 1], 100001, dtype) for i in range(2)]
    wants = [want(a) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [call(a) for a in cases]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    for a, s, out, graph in zip(cases, streams, outs, graphs):
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                call(a, out=out)
    for again in range(2):
        if again:  # the other's inputs of the same shape
            for a, b in zip(cases, [{k: v.clone() for k, v in a.items() if torch.is_tensor(v)}
                                    for a in reversed(cases)]):
                for k, v in b.items():
                    a[k].copy_(v)
            wants = wants[::-1]
        for out in outs:
            out[0].fill_(-7)
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(4):
                    graph.replay()
        torch.cuda.synchronize()
        for (tokens, accepted), (t, n) in zip(outs, wants):
            assert np.array_equal(tokens.cpu().numpy(), t) and np.array_equal(accepted.cpu().numpy(), n)
    no_error()
