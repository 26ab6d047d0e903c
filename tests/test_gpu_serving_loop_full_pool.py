"""The serving loop where the pool has too few pages: sequences that get none sit the step
out, their cached rows and those that others share with them stay as they are byte for byte,
and they go on once others have given pages back."""
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import DEV, i32, no_error
from tests.test_gpu_serving_loop import D, G, HKV, Loop

pytestmark = pytest.mark.gpu


class FullPool(Loop):
    def pool(self):
        return [{name: getattr(kv, name).view(torch.uint8).clone()
                 for name in ("k", "v", "k_scale", "v_scale", "k_bs", "v_bs")
                 if getattr(kv, name) is not None} for kv in self.kv.caches]

    def step(self, asked):
        """asked[s] new positions (the last token and drafted ones), as far as there are
        pages; how many each sequence got."""
        before, L = self.pool(), self.len.tolist()
        want = plain.reserve(self.refs.tolist(), self.table.tolist(), L,
                             [a + m for a, m in zip(L, asked)], self.ps)
        kv_len = self.len
        grown, src, dst = bs.attn_skip_pages_reserve(self.refs, self.table, kv_len,
                                                     kv_len + i32(asked), self.ps)
        assert self.refs.tolist() == want[0] and self.table.tolist() == want[1]
        assert [x.tolist() for x in (grown, src, dst)] == list(want[2:5])
        bs.attn_skip_kv_copy_pages(self.kv, src, dst)
        n = (grown - kv_len).tolist()
        cu = i32(np.concatenate(([0], np.cumsum(n))))
        self.len = grown
        for i, kv in enumerate(self.kv.caches):
            k, v = self.rows(sum(n)), self.rows(sum(n))
            bs.attn_skip_kv_append(kv, k, v, cu, grown, self.table)
            ks, vs = bs.attn_skip_kv_gather(kv, cu, kv_len, self.table, sum(n))
            at = 0
            for s, m in enumerate(n):
                a, b = self.past[s][i]
                self.past[s][i] = (torch.cat((a, ks[at:at + m])), torch.cat((b, vs[at:at + m])))
                at += m
        # Pages that no sequence writes into are what they were: all but the new ones (free
        # before), the copies, and the last pages of those that grew within theirs.
        written = set(want[4])
        for s, m in enumerate(n):
            if m:
                written |= set(want[1][s][L[s] // self.ps:plain.up(L[s] + m, self.ps)])
        same = torch.tensor([p for p in range(len(want[0])) if p not in written], device=DEV)
        for one, was in zip(self.pool(), before):
            for name, x in one.items():
                assert torch.equal(x[same], was[name][same]), name
        return n, cu

    def attend(self, cu, n):
        """As in the loop, which has no empty chunks: the same bound."""
        q = torch.randn(sum(n), HKV * G, D, device=DEV, generator=self.gen).to(torch.bfloat16)
        for i, kv in enumerate(self.kv.caches):
            o, _, _ = bs.attn_skip_chunk_paged(kv, q, cu, max(n), self.len, int(self.len.max()),
                                               self.table, torch.zeros(len(n), device=DEV))
            at = 0
            for s, m in enumerate(n):
                if not m:
                    continue
                k, v = (x.double() for x in self.past[s][i])
                L = len(k)
                x = torch.einsum("thgd,lhd->thgl", q[at:at + m].double().reshape(m, HKV, G, D), k)
                hide = torch.arange(L, device=DEV) > torch.arange(L - m, L, device=DEV)[:, None]
                x = (x / math.sqrt(D)).masked_fill(hide[:, None, None], -math.inf)
                want = torch.einsum("thgl,lhd->thgd", x.softmax(-1), v).reshape(m, HKV * G, D)
                assert (o[at:at + m].double() - want).abs().max() < 5 * 2.0 ** -7
                at += m

    def verify(self, n):
        """The drafts of the sequences that take part; the batch goes back to what they accept."""
        took = [s for s, m in enumerate(n) if m]
        drafts = [n[s] - 1 for s in took]
        V, total = 500, sum(drafts)
        target = torch.softmax(2 * torch.randn(total + len(took), V, device=DEV, generator=self.gen), -1)
        x = torch.randint(0, V, (total,), device=DEV, generator=self.gen).to(torch.int32)
        u, us = (torch.rand(m, device=DEV, generator=self.gen) for m in (total, len(took)))
        cu = i32(np.concatenate(([0], np.cumsum(drafts))))
        _, accepted = bs.attn_skip_verify_drafts(target, x, cu, max(drafts), u / 50, us)
        kept = self.len.index_add(0, torch.tensor(took, device=DEV), accepted - i32(drafts))
        bs.attn_skip_pages_fork(self.refs, self.table, self.len, kept, self.ps)
        self.len = kept
        self.past = [[(k[:L], v[:L]) for k, v in p] for p, L in zip(self.past, kept.tolist())]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "nvfp4"])
def test_a_loop_whose_pages_run_out(fmt):
    z = FullPool(fmt, 16, 10, 8, seed=11)
    z.start(3)
    z.grow([40, 21, 5])  # 3 + 2 + 1 pages
    z.check()
    # Seven sequences: the first prompt with three followers that share a partly filled page,
    # the second with two, the third alone.
    z.fork([0, 0, 0, 1, 1, 2, 2], [40, 40, 40, 21, 21, 5, 5])
    z.check()
    refused = served = 0
    for step in range(7):
        asked = [z.r.choice((1, 4, 6, 18)) for _ in range(len(z.past))]
        n, cu = z.step(asked)
        refused += sum(m == 0 for m in n)
        served += sum(m > 0 for m in n)
        z.check()
        if sum(n):
            z.attend(cu, n)
            z.verify(n)
            z.check()
        if step == 4:  # two sequences end; the others go on, in another order
            order = [4, 3, 2, 1, 0]
            z.fork(order, [int(z.len[s]) for s in order])
            z.check()
    assert refused > 3 and served > 3
    # All but one end: it gets what it asks for.
    z.fork([3], [int(z.len[3])])
    n, cu = z.step([30])
    assert n == [30]
    z.check()
    z.attend(cu, n)
    bs.attn_skip_pages_fork(z.refs, z.table, z.len, i32([0]), z.ps)
    assert int(z.refs.abs().sum()) == 0
    no_error()


def test_nobody_gets_a_page():
    """Every sequence shares its last page and the pool is full: the step writes nothing."""
    z = FullPool("e4m3", 16, 3, 4, seed=5)
    z.start(1)
    z.grow([40])
    z.fork([0, 0, 0], [40, 40, 39])
    n, _ = z.step([1, 5, 2])
    assert n == [0, 0, 0]
    z.check()
    # A chunk that its pages take: one that has the last page to itself.
    z.fork([1], [40])
    n, cu = z.step([8])
    assert n == [8]
    z.attend(cu, n)
    z.check()
    no_error()
