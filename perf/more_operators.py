"""Cases, plain forms and 64-bit values of the operators that keep a paged cache in
a serving loop, and of the check of drafted tokens.

Five operators around one paged cache (its formats: bf16 rows; E4M3 rows; NVFP4
rows) and the page tables of a batch:

* ``reserve``: pages for the tokens that are about to come, the lowest free ones,
  and a page of its own for a sequence that would write into a shared one;
* ``fork``: the sequences of the next batch take over pages of this one's (a fork, a
  reordering of beams, a truncation, the end of a sequence), reference counts kept;
* ``copy``: whole pages copied, in every layer at once;
* ``compact``: the rows that are kept move together, in every layer at once;
* ``verify``: drafted tokens accepted or replaced by rejection sampling against the
  target's probabilities.

``own`` false computes them with elementary torch operations, ``own`` true with the
library's entry points.
"""
import math
import random

import torch

own = False

D = 128  # head size


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # One conversation, four drafted tokens: pure latency.
        dict(name="verify 1 seq", op="verify", n_seq=1, draft=4, V=32000, dtype="fp32", probs=True,
             sharp=2.5, noise=0.7, cut=False, lens=0),
        # A batch whose drafts come from a look-up (no distribution), odd vocabulary, bf16, tails cut.
        dict(name="verify 48 look-up", op="verify", n_seq=48, draft=7, V=50001, dtype="bf16",
             probs=False, sharp=3.0, noise=0.5, cut=True, lens=1),
        # A large batch with a draft model, a large vocabulary.
        dict(name="verify 256 seqs", op="verify", n_seq=256, draft=5, V=128000, dtype="fp32",
             probs=True, sharp=2.5, noise=0.7, cut=False, lens=2),
        # A decode step of 64 sequences: few need a page, some write into a forked one.
        dict(name="reserve decode 64", op="reserve", n_seq=64, max_new=1, max_kv=4096, page=16,
             pages=20000, share=0.25, lens=3),
        # A wave of prompts enters a large pool.
        dict(name="reserve prompts 1000", op="reserve", n_seq=1000, max_new=1531, max_kv=2200,
             page=16, pages=262144, share=0.1, lens=4),
        # Eight prompts, four beams each: the beams go on from one another.
        dict(name="fork beams 8x4", op="fork", n_seq=32, n_new=32, max_kv=2500, page=16,
             mode="beams", group=4, lens=5),
        # A large batch of long sequences is rebuilt: some end, some fork, some lose drafted tokens.
        dict(name="fork 512 x 32768", op="fork", n_seq=512, n_new=512, max_kv=32768, page=16,
             mode="mixed", group=8, lens=6),
        # Four beams write on: their last pages in one layer.
        dict(name="copy 4 pages e4m3", op="copy", fmt="e4m3", pairs=4, gaps=0, layers=1, pool=40,
             page=16, Hkv=8),
        # A batch forks: last pages of 96 sequences in 32 layers, entries of others that need none.
        dict(name="copy 96 pages x 32", op="copy", fmt="bf16", pairs=96, gaps=32, layers=32,
             pool=224, page=64, Hkv=8),
        # The accepted path of a drafted tree moves up behind the cached rows.
        dict(name="compact path e4m3", op="compact", fmt="e4m3", kind="path", n_seq=16, max_kv=2000,
             keep=4, layers=32, page=64, Hkv=8, per_head=False, lens=7),
        # A long sequence keeps its first tokens and a window of its last.
        dict(name="compact window bf16", op="compact", fmt="bf16", kind="window", n_seq=1,
             max_kv=32768, keep=8192, layers=8, page=64, Hkv=8, per_head=False, lens=0),
        # Every head of ragged sequences keeps its own half of the rows, in other pages.
        dict(name="compact heads nvfp4", op="compact", fmt="nvfp4", kind="scattered", n_seq=9,
             max_kv=5001, keep=2500, layers=4, page=16, Hkv=4, per_head=True, lens=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("verify", "verify", "reserve", "fork", "copy", "compact", "compact"))
    c = dict(op=op, lens=rng.randrange(1, 1 << 20))
    if op == "verify":
        c["V"], c["draft"] = _log(rng, 1000, 200000), rng.randint(0, 16)
        rows = (256 * 6 * 128000) // (c["V"] * (c["draft"] + 1))
        c["n_seq"] = _log(rng, 1, max(1, min(512, rows)))
        c["dtype"], c["probs"] = rng.choice(("fp32", "bf16")), rng.random() < 0.7
        c["sharp"], c["noise"] = rng.choice((1.0, 2.5, 4.0)), rng.choice((0.1, 0.7, 2.0))
        c["cut"] = rng.random() < 0.3
    elif op == "reserve":
        c["n_seq"], c["page"] = _log(rng, 1, 1000), rng.choice((16, 32, 64, 128, 256))
        c["max_new"] = rng.choice((1, rng.randint(2, 9), _log(rng, 10, 1531)))
        c["max_kv"] = c["max_new"] + _log(rng, 16, 8192)
        while c["n_seq"] * c["max_kv"] > 1 << 22:
            c["n_seq"] = c["n_seq"] // 2 + 1
        # Sometimes too few pages for all.
        want = c["n_seq"] * (-(-c["max_kv"] // c["page"]))
        c["pages"] = min(262144, int(want * rng.choice((0.9, 1.1, 2.0))) + 3)
        c["share"] = rng.choice((0.0, 0.25, 0.6))
    elif op == "fork":
        c["n_seq"], c["page"] = _log(rng, 1, 512), rng.choice((16, 32, 64, 128, 256))
        c["max_kv"] = _log(rng, 16, 32768)
        c["mode"], c["group"] = rng.choice(("beams", "mixed", "cut")), rng.randint(2, 9)
        c["n_new"] = c["n_seq"] if c["mode"] == "cut" else _log(rng, 1, 512)
    else:
        c["fmt"], c["Hkv"] = rng.choice(("bf16", "e4m3", "nvfp4")), rng.choice((1, 2, 3, 4, 8))
        c["page"], c["layers"] = rng.choice((16, 32, 64, 128, 256)), rng.choice((1, 2, 5, 32, 40))
        size = 2 * c["Hkv"] * c["layers"] * _row_bytes(c["fmt"])  # of a token
        if op == "copy":
            c["pairs"] = _log(rng, 1, max(1, min(512, (1 << 29) // (size * c["page"]))))
            c["gaps"] = rng.randrange(0, 40)
            c["pool"] = 2 * c["pairs"] + rng.randrange(1, 30)
        else:
            c["kind"] = rng.choice(("path", "window", "scattered"))
            c["max_kv"] = _log(rng, 32, 32768)
            c["n_seq"] = _log(rng, 1, max(1, min(64, (1 << 29) // (size * c["max_kv"]))))
            while c["layers"] > 1 and c["n_seq"] * c["max_kv"] * size > 1 << 30:
                size = size // c["layers"]
                c["layers"] = c["layers"] // 2
                size *= c["layers"]
            c["keep"] = (rng.randint(1, 7) if c["kind"] == "path"
                         else rng.randint(1, max(1, c["max_kv"] // 2 - 8)))
            c["per_head"] = c["kind"] == "scattered" and rng.random() < 0.5
    return c


def _row_bytes(fmt):
    return {"bf16": 2 * D, "e4m3": D + 1, "nvfp4": D // 2 + D // 16 + 1}[fmt]


SINK, TREE = 4, 16  # first tokens that a window keeps; rows of a drafted tree


def _host(case):
    """The lengths and choices of a case, from its own seed (not the inputs')."""
    r = random.Random(case.get("lens", 0) + 17)
    n, out = case.get("n_seq", 0), {}
    if case["op"] == "verify":
        out["n"] = [r.randint(0, case["draft"]) if case["lens"] else case["draft"] for _ in range(n)]
        out["n"][r.randrange(n)] = case["draft"]
    elif case["op"] == "reserve":
        new = [r.randint(1, case["max_new"]) for _ in range(n)]
        new[r.randrange(n)] = case["max_new"]
        old = [r.randint(0, case["max_kv"] - m) for m in new]
        out["old"], out["new"] = old, [a + m for a, m in zip(old, new)]
    elif case["op"] == "fork":
        L = [r.randint(max(1, case["max_kv"] // 2), case["max_kv"]) for _ in range(n)]
        L[r.randrange(n)] = case["max_kv"]
        g = case["group"]
        if case["mode"] == "beams":
            for s in range(n):  # beams of a group are as long as one another
                L[s] = L[s - s % g]
        m = case["n_new"]
        if case["mode"] == "cut":  # in place: drafted tokens go, some sequences end
            out["parent"], out["len"] = None, [0 if r.random() < 0.1 else max(0, x - r.randint(0, 9))
                                               for x in L]
        elif case["mode"] == "beams":
            out["parent"] = [min(n - 1, min(d, n - 1) // g * g + r.randrange(g)) for d in range(m)]
            out["len"] = [L[p] for p in out["parent"]]
        else:
            out["parent"] = [-1 if x < 0.1 else min(d, n - 1) if x < 0.6 else r.randrange(n)
                             for d, x in ((d, r.random()) for d in range(m))]
            out["len"] = [0 if p < 0 else max(0, L[p] - r.choice((0, 0, r.randint(1, 9))))
                          for p in out["parent"]]
        out["old"] = L
    elif case["op"] == "compact":
        L, keep, start = [], [], []
        for s in range(n):
            x = case["max_kv"] if not case["lens"] or s == 0 else r.randint(
                max(1, case["max_kv"] // 2), case["max_kv"])
            k = min(case["keep"] if s == 0 else r.randint(1, case["keep"]), max(1, x // 2 - 8))
            if case["kind"] == "path":
                k = min(k, x // 2)
                t = min(x, max(2 * k, TREE))
                start.append(x - t)
                keep.append(sorted(x - t + i for i in r.sample(range(k, t), k)))
            elif case["kind"] == "window":
                start.append(0)
                keep.append(list(range(min(SINK, x - k))) + list(range(x - k, x)))
            else:
                start.append(0)
                keep.append(k)  # how many; which ones come from the inputs' seed
            L.append(x)
        out.update(len=L, keep=keep, start=start)
    return out


def work(case):
    h = _host(case)
    if case["op"] == "verify":
        # A row of the target's for each sequence, one of the draft's where a token may be
        # rejected, and three values, a token and a random number for each drafted token.
        e = 4 if case["dtype"] == "fp32" else 2
        n, drafts = case["n_seq"], sum(h["n"])
        rows = n + (sum(1 for x in h["n"] if x) if case["probs"] else 0)
        return dict(bytes=rows * case["V"] * e + drafts * (2 * e + 8) + n * 4 * (case["draft"] + 4),
                    flops=2 * rows * case["V"])
    ps = case["page"]
    up = lambda x: -(-x // ps)
    if case["op"] == "reserve":
        new = sum(up(b) - up(a) for a, b in zip(h["old"], h["new"]))
        return dict(bytes=4 * (case["pages"] + 2 * new + 5 * case["n_seq"]), flops=0)
    if case["op"] == "fork":
        old, new = sum(map(up, h["old"])), sum(map(up, h["len"]))
        ids = abs(old - new) if h["parent"] is None else old + 2 * new
        return dict(bytes=4 * (ids + 2 * abs(old - new) + 2 * case["n_seq"] + 2 * case["n_new"]),
                    flops=0)
    size = 2 * case["Hkv"] * case["layers"] * _row_bytes(case["fmt"])
    if case["op"] == "copy":
        return dict(bytes=2 * case["pairs"] * ps * size + 8 * (case["pairs"] + case["gaps"]), flops=0)
    if case["kind"] == "scattered":
        rows = sum(h["keep"])
    else:  # rows that stay where they are cost nothing
        rows = sum(k != st + j for ks, st in zip(h["keep"], h["start"]) for j, k in enumerate(ks))
    return dict(bytes=2 * rows * size + 4 * rows * (case["Hkv"] if case["per_head"] else 1), flops=0)


# ------------------------------------------------------------------ inputs --
def _gen(seed, tag):
    return torch.Generator(device="cuda").manual_seed((int(seed) * 1000003 + tag) & (2**62 - 1))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _cu(n):
    return torch.tensor([0] + list(n)).cumsum(0).to(device="cuda", dtype=torch.int32)


def _tables(lens, width, n_pages, gen):
    """Pages in random order for sequences of these lengths in pages; -1 elsewhere."""
    order = torch.randperm(n_pages, device="cuda", generator=gen).to(torch.int32)
    n = torch.tensor(lens).cuda()
    slot = (n.cumsum(0) - n)[:, None] + torch.arange(width, device="cuda")
    used = torch.arange(width, device="cuda") < n[:, None]
    return torch.where(used, order[slot.clamp(max=n_pages - 1)], torch.full_like(order[:1], -1)), used


def _count(table, used, n_pages):
    """How many used entries name each page."""
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    return refs.index_add_(0, torch.where(used, table, 0).flatten().long(),
                           used.flatten().to(torch.int32))


def _prepare_verify(case, seed):
    n, V = _host(case)["n"], case["V"]
    total, rows = sum(n), sum(n) + len(n)
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16

    def probs(x):
        p = torch.softmax(x, -1)
        if case["cut"]:  # tails cut, as by a nucleus
            p = torch.where(p < p.amax(-1, keepdim=True) / 500, torch.zeros_like(p), p)
            p = p / p.sum(-1, keepdim=True)
        return p

    z = torch.randn(rows, V, device="cuda", generator=_gen(seed, 1)) * case["sharp"]
    st = dict(case=case, target=probs(z).to(dt), cu=_cu(n), max_draft=case["draft"], draft=None)
    # Rows that have a drafted token: all but each sequence's last.
    last = torch.zeros(rows, dtype=torch.bool)
    last[torch.tensor(n).add(1).cumsum(0) - 1] = True
    keep = torch.nonzero(~last).flatten().cuda()
    z = z[keep]
    q = probs(z + case["noise"] * torch.randn(z.shape, device="cuda", generator=_gen(seed, 2)))
    del z
    if case["probs"]:  # drafted tokens are drawn from the draft's distribution
        e = torch.empty_like(q).exponential_(generator=_gen(seed, 3))
        st["drafted"] = (q / e).argmax(-1).to(torch.int32) if total else _i32([])
        st["draft"] = q.to(dt)
    else:  # a look-up: the likeliest token of a distribution near the target's
        st["drafted"] = q.argmax(-1).to(torch.int32) if total else _i32([])
    st["u_accept"] = torch.rand(total, device="cuda", generator=_gen(seed, 4))
    st["u_sample"] = torch.rand(len(n), device="cuda", generator=_gen(seed, 5))
    return st


def _prepare_reserve(case, seed):
    h, ps, n, N = _host(case), case["page"], case["n_seq"], case["pages"]
    width = -(-case["max_kv"] // ps)
    old = [-(-a // ps) for a in h["old"]]
    while sum(old) > N - 3:  # the pool holds what is cached
        i = old.index(max(old))
        old[i] //= 2
        h["old"][i] = min(h["old"][i], old[i] * ps)
    table, used = _tables(old, width, N, _gen(seed, 1))
    # Forks: a sequence shares all the pages of the one before it, as far as both reach.
    a = torch.tensor(h["old"])
    pick = torch.rand(n, generator=torch.Generator().manual_seed(int(seed) + 7)) < case["share"]
    src = torch.arange(n)
    for s in range(1, n):
        if pick[s] and h["old"][s - 1] > 0:
            src[s] = src[s - 1]
            grow = max(1, h["new"][s] - h["old"][s])
            a[s] = a[src[s]]
            h["new"][s] = min(int(a[s]) + grow, case["max_kv"])
    new = torch.maximum(torch.tensor(h["new"]), a)
    table, a = table[src.cuda()], a.to(device="cuda", dtype=torch.int32)
    used = torch.arange(width, device="cuda") < (-(-a // ps))[:, None]
    saved = torch.cat((_count(table, used, N), table.flatten().to(torch.int32)))
    live = saved.clone()
    return dict(case=case, saved=saved, live=live, refs=live[:N], table=live[N:].view(n, width),
                old=a, new=new.to(device="cuda", dtype=torch.int32))


def _prepare_fork(case, seed):
    h, ps = _host(case), case["page"]
    width = -(-case["max_kv"] // ps)
    old = [-(-a // ps) for a in h["old"]]
    N = sum(old) + 5
    table, used = _tables(old, width, N, _gen(seed, 1))
    if case["mode"] == "beams":  # a group's beams share the prompt, about two thirds of their pages
        g, n = case["group"], case["n_seq"]
        first = torch.arange(n, device="cuda") // g * g
        shared = torch.arange(width, device="cuda") < (torch.tensor(old).cuda() * 2 // 3)[:, None]
        table = torch.where(shared, table[first], table)
    saved = _count(table, used, N)
    return dict(case=case, saved=saved, refs=saved.clone(), table=table, old=_i32(h["old"]),
                parent=None if h["parent"] is None else _i32(h["parent"]), len=_i32(h["len"]),
                out=None if h["parent"] is None else torch.full(
                    (case["n_new"], width), -1, dtype=torch.int32, device="cuda"))


def _pool(case, n_pages, seed):
    """The pools of the layers, pages filled: one tensor [layers, pages, ...] a part."""
    rows, g = (case["layers"], n_pages, case["Hkv"], case["page"]), _gen(seed, 9)

    def u8(lo, hi, *shape):
        return torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)

    pool = {}
    for w in ("k", "v"):
        if case["fmt"] == "bf16":
            pool[w] = torch.randn(*rows, D, dtype=torch.bfloat16, device="cuda", generator=g)
            continue
        if case["fmt"] == "e4m3":  # both signs, no NaN codes
            pool[w] = u8(0, 127, *rows, D) | (u8(0, 2, *rows, D) << 7)
        else:
            pool[w] = u8(0, 256, *rows, D // 2)
            pool[w + "_bs"] = u8(0, 127, *rows, D // 16)
        pool[w + "_scale"] = u8(110, 130, *rows)
    return pool


def _prepare_copy(case, seed):
    n, g = case["pool"], _gen(seed, 1)
    order = torch.randperm(n, device="cuda", generator=g).to(torch.int32)
    src, dst = order[:case["pairs"]], order[case["pairs"]:2 * case["pairs"]]
    none = torch.full((case["gaps"],), -1, dtype=torch.int32, device="cuda")
    mix = torch.randperm(case["pairs"] + case["gaps"], device="cuda", generator=g)
    return dict(case=case, src=torch.cat((src, none))[mix], dst=torch.cat((dst, none))[mix],
                pool=_pool(case, n, seed))


def _prepare_compact(case, seed):
    h, ps = _host(case), case["page"]
    old = [-(-x // ps) for x in h["len"]]
    scattered = case["kind"] == "scattered"
    count = h["keep"] if scattered else [len(k) for k in h["keep"]]
    more = [-(-c // ps) for c in count] if scattered else [0] * len(old)
    N, width = sum(old) + sum(more) + 3, max(old)
    table, _ = _tables(old + more, width, N, _gen(seed, 1))
    st = dict(case=case, table=table[:len(old)].contiguous(), cu=_cu(count), total=sum(count),
              start=_i32(h["start"]), out_table=None, pool=_pool(case, N, seed))
    if scattered:
        # Each head (or all alike) keeps a random subset, in order.
        st["out_table"] = table[len(old):].contiguous()
        heads, g = case["Hkv"] if case["per_head"] else 1, _gen(seed, 2)
        st["keep"] = torch.stack([torch.cat([
            torch.randperm(x, device="cuda", generator=g)[:c].sort().values
            for x, c in zip(h["len"], count)]) for _ in range(heads)]).to(torch.int32)
        if not case["per_head"]:
            st["keep"] = st["keep"][0]
    else:
        st["keep"] = _i32([k for ks in h["keep"] for k in ks])
    return st


def prepare(case, seed):
    st = dict(verify=_prepare_verify, reserve=_prepare_reserve, fork=_prepare_fork,
              copy=_prepare_copy, compact=_prepare_compact)[case["op"]](case, seed)
    if own and "pool" in st:  # the cache handles that a program keeps
        from block_sparse_attention_online_gb300 import binding
        st["kv"] = binding.PagedLayers([
            binding.PagedKV(case["fmt"], **{name: x[i] for name, x in st["pool"].items()})
            for i in range(case["layers"])])
    return st


# ------------------------------------------------------------- plain forms --
def _plain_verify(st):
    """Acceptance tests and the cumulative sums in 64 bits: whole tokens come out."""
    cu, n_max, p = st["cu"].long(), st["max_draft"], st["target"]
    dev, n_seq, V = p.device, len(cu) - 1, p.shape[1]
    n = cu[1:] - cu[:-1]
    i = torch.arange(n_max, device=dev)
    have = i < n[:, None]
    accepted = torch.zeros(n_seq, dtype=torch.int64, device=dev)
    x = torch.full((n_seq, n_max), -1, dtype=torch.int64, device=dev)
    if len(st["drafted"]):
        d = torch.where(have, cu[:-1, None] + i, 0)
        x = torch.where(have, st["drafted"].long()[d], -1)
        row = d + torch.where(have, torch.arange(n_seq, device=dev)[:, None], 0)
        px = p[row, x.clamp(min=0)].double()
        qx = torch.ones_like(px) if st["draft"] is None else st["draft"][d, x.clamp(min=0)].double()
        ok = have & (st["u_accept"][d].double() * qx < px)
        accepted = ok.to(torch.int64).cumprod(-1).sum(-1)
    rejected = accepted < n
    w = p[cu[:-1] + torch.arange(n_seq, device=dev) + accepted].double()
    if len(st["drafted"]):
        at = torch.where(rejected, cu[:-1] + accepted, 0)
        if st["draft"] is None:
            r = w.scatter(1, st["drafted"].long()[at][:, None], 0.0)
        else:
            r = (w - st["draft"][at].double()).clamp_(min=0.0)
        some = rejected & (r.sum(-1) > 0)
        w = torch.where(some[:, None], r, w)
    F = w.cumsum(-1)
    T = st["u_sample"].double()[:, None] * F[:, -1:]
    token = (F <= T).sum(-1).clamp(max=V - 1)
    out = torch.full((n_seq, n_max + 1), -1, dtype=torch.int64, device=dev)
    out[:, :n_max] = torch.where(i < accepted[:, None], x, -1)
    out.scatter_(1, accepted[:, None], token[:, None])
    return out.to(torch.int32), accepted.to(torch.int32)


def _plain_reserve(st):
    refs, table, a, b, ps = st["refs"], st["table"], st["old"], st["new"], st["case"]["page"]
    n, width, N, dev = len(a), table.shape[1], len(refs), refs.device
    first, last = (a + ps - 1) // ps, (b + ps - 1) // ps
    at = (a // ps).clamp(max=width - 1).long()[:, None]
    partial = (a % ps != 0) & (b > a)
    page = torch.where(partial, table.gather(1, at)[:, 0], -1).long()
    holders = torch.where(partial, refs[page.clamp(min=0)], 0)
    shared = holders > 1
    # Earlier sequences of the batch that write into the same shared page.
    s = torch.arange(n, device=dev)
    rank = ((page[:, None] == page) & shared & (s[:, None] > s)).sum(-1)
    cow = shared & (rank < holders - 1)
    need = cow.to(torch.int64) + last - first
    upto = need.cumsum(0)
    free = refs == 0
    k = free.to(torch.int64).cumsum(0) - 1  # number of a free page
    served = (upto <= k[-1] + 1) | ((need == 0) & ~shared)
    page_of = torch.zeros(N + 1, dtype=torch.int32, device=dev)
    page_of.scatter_(0, torch.where(free, k, N), torch.arange(N, device=dev, dtype=torch.int32))
    cow &= served
    begin = upto - need
    own_page = page_of[torch.where(cow, begin, N)]
    e = torch.arange(width, device=dev)
    mine = served[:, None] & (e >= first[:, None]) & (e < last[:, None])
    number = (begin + cow)[:, None] + e - first[:, None]
    table.copy_(torch.where(mine, page_of[torch.where(mine, number, N)], table))
    table.scatter_(1, at, torch.where(cow, own_page, table.gather(1, at)[:, 0])[:, None])
    taken = torch.where(served, upto, 0).amax()
    refs.copy_(torch.where(free & (k < taken), 1, refs))
    refs.index_add_(0, torch.where(cow, page, 0), -cow.to(torch.int32))
    none = torch.full_like(own_page, -1)
    return (torch.where(served, b, a), torch.where(cow, page.to(torch.int32), none),
            torch.where(cow, own_page, none))


def _plain_fork(st):
    refs, table, a, b, ps = st["refs"], st["table"], st["old"], st["len"], st["case"]["page"]
    e = torch.arange(table.shape[1], device=refs.device)
    used = e < ((a + ps - 1) // ps)[:, None]
    kept = e < ((b + ps - 1) // ps)[:, None]
    refs.index_add_(0, torch.where(used, table, 0).flatten().long(),
                    -used.flatten().to(torch.int32))
    if st["parent"] is None:
        new = out = table
    else:
        new, out = table[st["parent"].clamp(min=0).long()], st["out"]
        out.copy_(torch.where(kept, new, out))
    refs.index_add_(0, torch.where(kept, new, 0).flatten().long(), kept.flatten().to(torch.int32))
    return out


def _plain_copy(st):
    # Entries without a page copy one that no pair names onto itself.
    src, dst = st["src"].long(), st["dst"].long()
    none = src < 0
    spare = _spare(st)
    src, dst = torch.where(none, spare, src), torch.where(none, spare, dst)
    for part in st["pool"].values():
        for x in part:
            x[dst] = x[src]


def _spare(st):
    """A page that no pair names."""
    n = st["case"]["pool"]
    named = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    for x in (st["src"], st["dst"]):
        named[torch.where(x < 0, n, x).long()] = 1
    return named[:n].argmin()


def _of_rows(cu, total):
    """Per kept row: its sequence and its number in it."""
    t = torch.arange(total, device=cu.device, dtype=torch.int32)
    s = torch.searchsorted(cu[1:], t, right=True)
    return s, t - cu[s]


def _plain_compact(st):
    ps, keep = st["case"]["page"], st["keep"]
    s, j = _of_rows(st["cu"], st["total"])
    to = st["start"][s] + j
    out = st["table"] if st["out_table"] is None else st["out_table"]
    p1, r1 = out[s, (to // ps).long()].long(), (to % ps).long()
    p0, r0 = st["table"][s, (keep // ps).long()].long(), (keep % ps).long()
    if keep.dim() == 2:
        h = torch.arange(keep.shape[0], device=keep.device)[:, None]
        a, b = (p0, h, r0), (p1.expand_as(p0), h, r1.expand_as(r0))
    else:
        a, b = (p0, slice(None), r0), (p1, slice(None), r1)
    for part in st["pool"].values():
        for x in part:
            x[b] = x[a]


# --------------------------------------------------------------------- run --
def _contents(st):
    """The pool: E4M3 codes as the values that they stand for, NVFP4 codes by their bytes."""
    out = []
    for name, x in sorted(st["pool"].items()):
        e4m3 = name.endswith("_bs") or (st["case"]["fmt"] == "e4m3" and name in ("k", "v"))
        out.append(x.view(torch.float8_e4m3fn) if e4m3 else x)
    return out


def run(state):
    st, op = state, state["case"]["op"]
    # The counts and tables as the call finds them: what it changes is put back first.
    if op == "reserve":
        st["live"].copy_(st["saved"])
    elif op == "fork":
        st["refs"].copy_(st["saved"])
    if own:
        from block_sparse_attention_online_gb300 import binding as bs
        if op == "verify":
            return bs.attn_skip_verify_drafts(st["target"], st["drafted"], st["cu"],
                                              st["max_draft"], st["u_accept"], st["u_sample"],
                                              draft=st["draft"])
        if op == "reserve":
            got = bs.attn_skip_pages_reserve(st["refs"], st["table"], st["old"], st["new"],
                                             st["case"]["page"])
        elif op == "fork":
            got = bs.attn_skip_pages_fork(st["refs"], st["table"], st["old"], st["len"],
                                          st["case"]["page"], parent=st["parent"],
                                          out_table=st["out"])
        elif op == "copy":
            bs.attn_skip_kv_copy_pages(st["kv"], st["src"], st["dst"])
        else:
            bs.attn_skip_kv_compact(st["kv"], st["keep"], st["cu"], st["table"],
                                    start=st["start"], out_table=st["out_table"])
    elif op == "verify":
        return _plain_verify(st)
    else:
        got = dict(reserve=_plain_reserve, fork=_plain_fork, copy=_plain_copy,
                   compact=_plain_compact)[op](st)
    if op == "reserve":
        return (*got, st["refs"], st["table"])
    if op == "fork":
        return got, st["refs"]
    return _contents(st)


# ------------------------------------------------------------------- exact --
def _x_verify(st):
    """One sequence at a time, from the definition."""
    cu, V = st["cu"].tolist(), st["target"].shape[1]
    out = torch.full((len(cu) - 1, st["max_draft"] + 1), -1, dtype=torch.int32)
    acc = torch.zeros(len(cu) - 1, dtype=torch.int32)
    x, ua, us = st["drafted"].tolist(), st["u_accept"].tolist(), st["u_sample"].tolist()
    for s in range(len(cu) - 1):
        n, w = cu[s + 1] - cu[s], None
        for i in range(n):
            d = cu[s] + i
            p = st["target"][d + s].double()
            q = torch.zeros_like(p)
            if st["draft"] is None:
                q[x[d]] = 1.0
            else:
                q = st["draft"][d].double()
            if ua[d] * q[x[d]].item() < p[x[d]].item():
                out[s, i] = x[d]
                acc[s] += 1
                continue
            w = torch.maximum(p - q, torch.zeros_like(p))
            if not w.any():
                w = p
            break
        if w is None:
            w = st["target"][cu[s + 1] + s].double()
        F = w.cumsum(0)
        t = torch.searchsorted(F, us[s] * F[-1], right=True)
        out[s, int(acc[s])] = min(int(t), V - 1)
    return out.cuda(), acc.cuda()


def _x_reserve(st):
    """One sequence after the other, as a program on the host would."""
    refs, table = st["refs"].tolist(), [r for r in st["table"].tolist()]
    a, b, ps = st["old"].tolist(), st["new"].tolist(), st["case"]["page"]
    holders = list(refs)  # of shared pages, as the sequences go on
    free = [p for p, r in enumerate(refs) if r == 0]
    at, full = 0, False
    got, src, dst = [], [], []
    for s in range(len(a)):
        e, page = a[s] // ps, -1
        if a[s] % ps and b[s] > a[s]:
            page = table[s][e]
        shared = page >= 0 and refs[page] > 1
        cow = shared and holders[page] > 1
        first, last = -(-a[s] // ps), -(-b[s] // ps)
        need = last - first + cow
        if cow:
            holders[page] -= 1
        full = full or (need > 0 and at + need > len(free))
        if full and (need > 0 or shared):
            got.append(a[s]), src.append(-1), dst.append(-1)
            continue
        got.append(b[s])
        src.append(page if cow else -1)
        dst.append(free[at] if cow else -1)
        if cow:
            table[s][e] = free[at]
            at += 1
        for f in range(first, last):
            table[s][f] = free[at]
            at += 1
    new = [r for r in refs]
    for p in free[:at]:
        new[p] = 1
    for p in src:
        if p >= 0:
            new[p] -= 1
    return _i32(got), _i32(src), _i32(dst), _i32(new), _i32(table)


def _x_fork(st):
    refs, table = st["refs"].tolist(), st["table"].cpu()
    a, b, ps = st["old"].tolist(), st["len"].tolist(), st["case"]["page"]
    for s, L in enumerate(a):
        for f in table[s, :-(-L // ps)].tolist():
            refs[f] -= 1
    parent = None if st["parent"] is None else st["parent"].tolist()
    out = (table if parent is None else st["out"].cpu()).clone()
    for d, L in enumerate(b):
        n = -(-L // ps)
        if parent is not None and n:
            out[d, :n] = table[parent[d], :n]
        for f in out[d, :n].tolist():
            refs[f] += 1
    return out.cuda(), _i32(refs)


def _x_copy(st):
    pairs = [(a, b) for a, b in zip(st["src"].tolist(), st["dst"].tolist()) if a >= 0]
    got = []
    for x in _contents(st):
        y = x.clone()
        for a, b in pairs:
            y[:, b].copy_(x[:, a])
        got.append(y)
    return got


def _x_compact(st):
    """One sequence and head at a time, through its rows in a row."""
    case, cu, ps = st["case"], st["cu"].tolist(), st["case"]["page"]
    out = st["table"] if st["out_table"] is None else st["out_table"]
    start, got = st["start"].tolist(), []
    keep = st["keep"] if st["keep"].dim() == 2 else st["keep"].expand(case["Hkv"], -1)
    moves = []
    for s in range(len(cu) - 1):
        to = torch.arange(start[s], start[s] + cu[s + 1] - cu[s], device="cuda")
        for h in range(case["Hkv"]):
            k = keep[h, cu[s]:cu[s + 1]].long()
            moves.append((h, out[s, to // ps].long(), to % ps, st["table"][s, k // ps].long(), k % ps))
    for x in _contents(st):
        y = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x).clone()
        z = y.clone()
        for h, to_page, to_row, page, row in moves:
            z[:, to_page, h, to_row] = y[:, page, h, row]
        got.append(z.view(x.dtype))
    return got


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return dict(verify=_x_verify, reserve=_x_reserve, fork=_x_fork, copy=_x_copy,
                compact=_x_compact)[case["op"]](st)
