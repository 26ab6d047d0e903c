"""The paged-cache calls as a serving loop makes them: prompts enter, sequences fork, get
pages for drafted tokens, attend, have drafts checked, and go back to what was accepted;
rows are dropped, sequences end.  After every step each sequence's cached rows and its
attention are those of a history kept on the side."""
import math
import random

import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import pages_plain as plain
from tests.test_gpu_pages import DEV, i32, no_error

pytestmark = pytest.mark.gpu
D, LAYERS, HKV, G = 128, 2, 2, 4


class Loop:
    """The loop's state: a pool per layer, refs, tables, lengths; and the histories."""

    def __init__(self, fmt, ps, n_pages, width, seed):
        self.ps, self.r = ps, random.Random(seed)
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.kv = bs.PagedLayers([bs.PagedKV.empty(fmt, n_pages, ps, HKV) for _ in range(LAYERS)])
        for kv in self.kv.caches:  # unwritten pages hold NaN: nothing may come of them
            for x in (kv.k, kv.v):
                x.fill_(float("nan") if fmt == "bf16" else 0)
            if fmt != "bf16":
                kv.k_scale.fill_(255), kv.v_scale.fill_(255)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        self.width = width
        self.table, self.len = i32(np.zeros((0, width))), i32([])
        self.past = []  # per sequence, per layer: (k, v) rows [len, HKV, D] as stored

    def rows(self, n):
        return torch.randn(n, HKV, D, device=DEV, generator=self.gen).to(torch.bfloat16)

    def grow(self, n):
        """n[s] new positions, their rows written in every layer."""
        new = self.len + i32(n)
        got, src, dst = bs.attn_skip_pages_reserve(self.refs, self.table, self.len, new, self.ps)
        assert torch.equal(got, new)
        bs.attn_skip_kv_copy_pages(self.kv, src, dst)
        cu = i32(np.concatenate(([0], np.cumsum(n))))
        start = self.len
        self.len = got
        for i, kv in enumerate(self.kv.caches):
            k, v = self.rows(sum(n)), self.rows(sum(n))
            bs.attn_skip_kv_append(kv, k, v, cu, self.len, self.table)
            ks, vs = bs.attn_skip_kv_gather(kv, cu, start, self.table, sum(n))
            at = 0
            for s, m in enumerate(n):
                p = self.past[s][i]
                self.past[s][i] = (torch.cat((p[0], ks[at:at + m])), torch.cat((p[1], vs[at:at + m])))
                at += m
        return cu

    def attend(self, cu, n):
        """Attention of the newest n[s] tokens against the histories, in 64 bits.  P rounded
        to 8 bits (half a step 2^-9 of 1) and the output to bf16 (2^-9 of itself): with
        values below 5 the error stays under 5 (2^-8 + 2^-8); scores add some 2^-13."""
        q = torch.randn(sum(n), HKV * G, D, device=DEV, generator=self.gen).to(torch.bfloat16)
        for i, kv in enumerate(self.kv.caches):
            o, _, _ = bs.attn_skip_chunk_paged(kv, q, cu, max(n), self.len, int(self.len.max()),
                                               self.table, torch.zeros(len(n), device=DEV))
            at = 0
            for s, m in enumerate(n):
                k, v = (x.double() for x in self.past[s][i])
                L = len(k)
                x = torch.einsum("thgd,lhd->thgl", q[at:at + m].double().reshape(m, HKV, G, D), k)
                hide = torch.arange(L, device=DEV) > torch.arange(L - m, L, device=DEV)[:, None]
                x = (x / math.sqrt(D)).masked_fill(hide[:, None, None], -math.inf)
                want = torch.einsum("thgl,lhd->thgd", x.softmax(-1), v).reshape(m, HKV * G, D)
                assert (o[at:at + m].double() - want).abs().max() < 5 * 2.0 ** -7
                at += m

    def check(self):
        """Rows are the histories', counts those of the tables."""
        n = self.len.tolist()
        refs = np.zeros(len(self.refs), dtype=int)
        for row, L in zip(self.table.tolist(), n):
            for p in row[:plain.up(L, self.ps)]:
                refs[p] += 1
        assert self.refs.tolist() == refs.tolist()
        if not sum(n):
            return
        cu = i32(np.concatenate(([0], np.cumsum(n))))
        for i, kv in enumerate(self.kv.caches):
            k, v = bs.attn_skip_kv_gather(kv, cu, None, self.table, sum(n))
            assert torch.equal(k, torch.cat([p[i][0] for p in self.past]))
            assert torch.equal(v, torch.cat([p[i][1] for p in self.past]))
        no_error()

    def fork(self, parent, new):
        self.table = bs.attn_skip_pages_fork(self.refs, self.table, self.len, i32(new), self.ps,
                                             parent=i32(parent))
        self.len = i32(new)
        self.past = [[(k[:L], v[:L]) for k, v in self.past[p]] if p >= 0
                     else [(self.rows(0), self.rows(0))] * LAYERS for p, L in zip(parent, new)]

    def start(self, n):
        """n empty sequences."""
        self.table = torch.full((n, self.width), -1, dtype=torch.int32, device=DEV)
        self.len = i32([0] * n)
        self.past = [[(self.rows(0), self.rows(0)) for _ in range(LAYERS)] for _ in range(n)]


@pytest.mark.parametrize("fmt,ps", [("bf16", 16), ("e4m3", 64), ("nvfp4", 16)])
def test_serving_loop(fmt, ps):
    z = Loop(fmt, ps, 400, 40, seed=ps)
    r = z.r
    z.start(3)
    n = [37, 5, 150]
    z.attend(z.grow(n), n)
    z.check()
    # Every prompt goes on in several samples, one of them cut back.
    z.fork([0, 0, 1, 2, 2, 2], [37, 37, 5, 150, 150, 149])
    z.check()
    for step in range(4):
        # Drafted tokens: the chunk is the last token and n of them.
        drafts = [r.randint(0, 5) for _ in range(6)]
        chunk = [d + 1 for d in drafts]
        z.attend(z.grow(chunk), chunk)
        z.check()
        V, total = 999, sum(drafts)
        target = torch.softmax(2 * torch.randn(total + 6, V, device=DEV, generator=z.gen), -1)
        last = np.cumsum(np.asarray(chunk)) - 1
        inner = torch.tensor(np.setdiff1d(np.arange(total + 6), last), dtype=torch.long, device=DEV)
        draft = (target[inner] + 0.3 / V) / 1.3
        x = (draft / torch.empty_like(draft).exponential_(generator=z.gen)).argmax(-1).to(torch.int32)
        ua, us = (torch.rand(m, device=DEV, generator=z.gen) for m in (total, 6))
        cu = i32(np.concatenate(([0], np.cumsum(drafts))))
        tokens, accepted = bs.attn_skip_verify_drafts(target, x, cu, 5, ua, us, draft=draft)
        t, a = plain.verify(target.double().cpu().numpy(), x.tolist(), cu.tolist(), 5, ua.tolist(),
                            us.tolist(), draft.double().cpu().numpy())
        assert np.array_equal(tokens.cpu().numpy(), t) and accepted.tolist() == a.tolist()
        # Back to what was accepted.
        keep = z.len - i32(drafts) + accepted
        bs.attn_skip_pages_fork(z.refs, z.table, z.len, keep, z.ps)
        z.len = keep
        z.past = [[(k[:L], v[:L]) for k, v in p] for p, L in zip(z.past, keep.tolist())]
        z.check()
    # A sequence drops what lies between its first four rows and its last twenty, in pages that it
    # has to itself: it alone goes on.
    z.fork([5], [int(z.len[5])])
    L = int(z.len[0])
    own = torch.full((1, 40), -1, dtype=torch.int32, device=DEV)
    got, _, _ = bs.attn_skip_pages_reserve(z.refs, own, i32([0]), i32([24]), z.ps)
    assert got.tolist() == [24]
    keep = list(range(4)) + list(range(L - 20, L))
    bs.attn_skip_kv_compact(z.kv, i32(keep), i32([0, 24]), z.table, out_table=own)
    bs.attn_skip_pages_fork(z.refs, z.table, z.len, i32([0]), z.ps)  # the old pages go back
    z.table, z.len = own, got
    z.past = [[(k[keep], v[keep]) for k, v in z.past[0]]]
    z.check()
    # A drafted tree of six rows whose path 1, 4 is accepted, moved up in place.
    z.grow([6])
    base = 24
    bs.attn_skip_kv_compact(z.kv, i32([base + 1, base + 4]), i32([0, 2]), z.table, start=i32([base]))
    keep = list(range(base)) + [base + 1, base + 4]
    bs.attn_skip_pages_fork(z.refs, z.table, z.len, i32([26]), z.ps)
    z.len = i32([26])
    z.past = [[(k[keep], v[keep]) for k, v in z.past[0]]]
    z.check()
    n = [1]
    z.attend(z.grow(n), n)
    z.check()
    # The end: every page is free again.
    bs.attn_skip_pages_fork(z.refs, z.table, z.len, i32([0]), z.ps)
    assert int(z.refs.abs().sum()) == 0
    no_error()
