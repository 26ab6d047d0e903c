"""The paged cache on the GPU (write, read back, attention of a chunk of new
tokens) against the plain 64-bit implementation."""
import numpy as np
import pytest
import torch

from block_sparse_attention_online_gb300 import binding as bs
from tests import paged_plain as plain
from tests.parity import MARGIN_BAND, compare_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMATS = ("bf16", "e4m3", "nvfp4")
ROW = {"bf16": 128, "e4m3": 128, "nvfp4": 64}


def filled_cache(fmt, n_pages, ps, Hkv):
    """A cache whose every byte reads as NaN (or as large garbage) until it is written."""
    kv = bs.PagedKV.empty(fmt, n_pages, ps, Hkv, device=DEV)
    for x in (kv.k, kv.v, kv.k_scale, kv.v_scale, kv.k_bs, kv.v_bs):
        if x is not None:
            x.view(torch.uint8).fill_(255)
    return kv


def tables(kv_lens, ps, g, spare=2, width=None):
    """A page table of distinct pages in random order; entries behind a
    sequence's last page hold ids that must not be read."""
    per = [-(-L // ps) for L in kv_lens]
    width = width or max(1, max(per))
    order = g.permutation(sum(per) + spare)
    t = np.full((len(kv_lens), width), 0x7fffffff, dtype=np.int32)
    at = 0
    for s, n in enumerate(per):
        t[s, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t).to(DEV), sum(per) + spare


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


def cu_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]))


def pool_rows(kv, table, s, L, which):
    """Positions 0 .. L-1 of a sequence from the pool tensors, float64 [L, Hkv, 128]."""
    t = table[s].cpu().numpy()
    pos = np.arange(L)
    page, slot = t[pos // kv.page_size], pos % kv.page_size

    def take(x):
        return x.cpu().numpy()[page, :, slot]
    x = getattr(kv, which)
    if kv.format == "bf16":
        return x.float().cpu().double().numpy()[page, :, slot]
    b = getattr(kv, which + "_bs")
    return plain.decode(kv.format, take(x), take(getattr(kv, which + "_scale")),
                        None if b is None else take(b))


def cache_of(fmt, kv_lens, ps, Hkv, seed, scale=1.0, sink=0.0):
    """A cache written by the library, its page table, and the rows it holds."""
    g = np.random.default_rng(seed)
    table, n_pages = tables(kv_lens, ps, g)
    kv = filled_cache(fmt, n_pages, ps, Hkv)
    total = sum(kv_lens)
    k = g.standard_normal((total, Hkv, 128)) * scale
    cu = np.concatenate([[0], np.cumsum(kv_lens)])
    for s, L in enumerate(kv_lens):  # a sink and some salient keys along a direction
        if L and sink:
            k[cu[s]] += sink
            k[cu[s]:cu[s] + L][g.random(L) < 0.01] += sink / 2
    k = torch.from_numpy(k).to(DEV, torch.bfloat16)
    v = torch.from_numpy(g.standard_normal((total, Hkv, 128)) * scale).to(DEV, torch.bfloat16)
    bs.attn_skip_kv_append(kv, k, v, cu_of(kv_lens), i32(kv_lens), table)
    bs.attn_skip_last_device_error()
    return kv, table


# ------------------------------------------------------------------ append --
def special_rows(g, n, Hkv, dtype):
    x = g.standard_normal((n, Hkv, 128)) * np.exp2(g.integers(-20, 20, (n, Hkv, 1)).astype(float))
    x = torch.from_numpy(x).to(dtype)
    flat = x.view(-1, 128)
    vals = [0.0, -0.0, 1e-45, 1e-38, 3.3e38, 448.0, 449.0, 2688.0, 1.0 / 3, 57345.0]
    for i, a in enumerate(vals):  # whole rows of one magnitude, and rows with one such element
        if 2 * i + 1 < len(flat):
            flat[2 * i] = a * torch.sign(flat[2 * i].float()).to(dtype)
            flat[2 * i + 1, i] = a
    if len(flat) > 26:
        flat[22, 3], flat[23, 127], flat[24, 0] = float("inf"), float("nan"), float("-inf")
        # Values half way between two codes of a row scale of 1: ties to even.
        flat[25] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 16).to(dtype)
        flat[26, :64] = (torch.arange(64) * 0.5 + 17).to(dtype)
    return x


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("chunks,before,ps,Hkv", [
    ((1,), (0,), 16, 1),
    ((3, 0, 17, 1), (5, 9, 0, 63), 16, 3),
    ((130, 64, 1), (0, 64, 127), 64, 2),
    ((390, 5), (379, 0), 384, 1),
    ((2500, 700), (3, 1000), 128, 8),  # the kernel's four rows a half warp
])
def test_append_writes_what_the_formats_define(fmt, dtype, chunks, before, ps, Hkv):
    g = np.random.default_rng(sum(chunks) + ps)
    lens = [a + b for a, b in zip(chunks, before)]
    table, n_pages = tables(lens, ps, g)
    kv = filled_cache(fmt, n_pages, ps, Hkv)
    total, tail = sum(chunks), 2  # rows behind the last sequence
    x = [special_rows(g, total + tail, Hkv, dtype) for _ in range(2)]
    # Rows of a fused projection: tokens further apart than their own row.
    fused = torch.zeros(total + tail, 3 * Hkv, 128, dtype=dtype, device=DEV)
    fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:] = x[0].to(DEV), x[1].to(DEV)
    bs.attn_skip_kv_append(kv, fused[:, Hkv:2 * Hkv], fused[:, 2 * Hkv:], cu_of(chunks), i32(lens),
                           table)
    bs.attn_skip_last_device_error()
    t, cu = table.cpu().numpy(), np.concatenate([[0], np.cumsum(chunks)])
    for which, src in zip("kv", x):
        pool = getattr(kv, which)
        want = {"codes": np.full(pool.shape, 255, np.uint8)}
        if fmt == "bf16":
            want = {"codes": np.full(pool.shape, -1, np.int16)}
            new = {"codes": src.to(torch.bfloat16).view(torch.int16).numpy()}
        else:
            want["scale"] = np.full(kv.k_scale.shape, 255, np.uint8)
            if fmt == "nvfp4":
                want["bs"] = np.full(kv.k_bs.shape, 255, np.uint8)
            new = plain.encode(fmt, src.double().numpy())
        for s, (c, L) in enumerate(zip(chunks, lens)):
            pos = np.arange(L - c, L)
            for name, w in want.items():
                w[t[s][pos // ps], :, pos % ps] = new[name][cu[s]:cu[s + 1]]
        got = {"codes": pool.view(torch.int16) if fmt == "bf16" else pool,
               "scale": getattr(kv, which + "_scale"), "bs": getattr(kv, which + "_bs")}
        for name, w in want.items():
            a = got[name].cpu().numpy()
            if fmt == "bf16":  # NaN payloads may differ
                f = got[name].view(torch.bfloat16).float().cpu().numpy()
                wf = torch.from_numpy(w).view(torch.bfloat16).float().numpy()
                assert (np.isnan(f) == np.isnan(wf)).all()
                a, w = np.where(np.isnan(f), 0, a), np.where(np.isnan(wf), 0, w)
            assert np.array_equal(a, w), f"{which} {name}: {(a != w).sum()} differ"


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_reports_bad_device_arguments_and_writes_the_rest(fmt):
    Hkv, ps = 2, 16
    kv = filled_cache(fmt, 6, ps, Hkv)
    before = [x.clone() for x in (kv.k, kv.v)]
    x = torch.randn(8, Hkv, 128, device=DEV).to(torch.bfloat16)
    # Sequence 0: a page id out of range; 1: a negative one; 2: a length beyond
    # the table; 3: sound; 4: a chunk longer than its cache (3 tokens, length 1).
    table = torch.tensor([[6, 0], [-1, 0], [1, 2], [3, 4], [5, 5]], dtype=torch.int32, device=DEV)
    bs.attn_skip_kv_append(kv, x, x, i32([0, 1, 2, 3, 5, 8]), i32([1, 1, 33, 17, 1]), table)
    with pytest.raises(bs.AttnSkipError) as e:
        bs.attn_skip_last_device_error()
    assert e.value.status == bs.ATTN_EINVAL
    bs.attn_skip_last_device_error()  # cleared
    changed = (kv.k.view(torch.uint8) != before[0].view(torch.uint8)).flatten(3).any(3)  # [page, head, slot]
    want = torch.zeros_like(changed)
    want[3, :, 15], want[4, :, 0], want[5, :, 0] = True, True, True
    assert torch.equal(changed, want)
    # Decreasing and out-of-range bounds: nothing is written, nothing faults.
    for cu in ([0, 9], [-1, 3], [5, 2]):
        bs.attn_skip_kv_append(kv, x, x, i32(cu), i32([8]), table[3:4].contiguous())
        after = kv.k.clone()
        try:
            bs.attn_skip_last_device_error()
        except bs.AttnSkipError as err:
            assert err.status == bs.ATTN_EINVAL
        assert torch.equal(after.view(torch.uint8), kv.k.view(torch.uint8))


# ------------------------------------------------------------------ gather --
def test_gather_reads_every_code_exactly():
    """Every E4M3 code under several row scales, every E2M1 pair under every
    block scale, in both output types."""
    Hkv, ps = 1, 16
    bytes_ = [17, 100, 120, 127, 134, 135, 200, 254, 255]
    kv = bs.PagedKV.empty("e4m3", 2, ps, Hkv, device=DEV)
    codes = np.arange(128, dtype=np.uint8)
    codes[127] = 0  # no E4M3 NaN codes in a cache
    kv.k.copy_(torch.from_numpy(np.broadcast_to(codes, (2, 1, ps, 128)).copy()))
    kv.v.copy_(torch.from_numpy(np.broadcast_to(codes | 128, (2, 1, ps, 128)).copy()))
    sc = np.resize(np.array(bytes_, np.uint8), 2 * ps).reshape(2, 1, ps)
    kv.k_scale.copy_(torch.from_numpy(sc))
    kv.v_scale.copy_(torch.from_numpy(sc))
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    for dt in (torch.bfloat16, torch.float32):
        k, v = bs.attn_skip_kv_gather(kv, i32([0, 27]), i32([3]), table, 27, dt)
        bs.attn_skip_last_device_error()
        rows = sc[::-1].reshape(-1)[3:30]
        for got, c in ((k, codes), (v, codes | 128)):
            want = plain.decode("e4m3", np.broadcast_to(c, (27, 128)), rows)
            want = torch.from_numpy(want).to(dt).double().numpy()  # overflow only at byte 254
            np.testing.assert_array_equal(got[:, 0].double().cpu().numpy(), want)
    kv = bs.PagedKV.empty("nvfp4", 2, ps, Hkv, device=DEV)
    g = np.random.default_rng(3)
    c = np.concatenate([np.arange(256)] * 8).astype(np.uint8).reshape(2, 1, ps, 64)
    b = g.integers(0, 127, (2, 1, ps, 8)).astype(np.uint8)
    s = g.integers(60, 190, (2, 1, ps)).astype(np.uint8)
    for x, y in ((kv.k, c), (kv.v, c), (kv.k_bs, b), (kv.v_bs, b), (kv.k_scale, s),
                 (kv.v_scale, s)):
        x.copy_(torch.from_numpy(y))
    for dt in (torch.bfloat16, torch.float32):
        k, v = bs.attn_skip_kv_gather(kv, i32([0, 32]), None, table, 32, dt)
        want = plain.decode("nvfp4", c[::-1].reshape(32, 64), s[::-1].reshape(32),
                            b[::-1].reshape(32, 8))
        np.testing.assert_array_equal(k[:, 0].double().cpu().numpy(), want)
        np.testing.assert_array_equal(v[:, 0].double().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,starts,ps,Hkv", [
    ((1,), None, 16, 1), ((5, 0, 33), (11, 3, 0), 16, 3), ((3000, 1), (77, 12), 256, 8),
    ((500, 9), (300, 380), 384, 1),
])
def test_gather_matches_the_pool(fmt, lens, starts, ps, Hkv):
    ends = [a + b for a, b in zip(lens, starts or (0,) * len(lens))]
    kv, table = cache_of(fmt, [max(1, e) for e in ends], ps, Hkv, 7)
    total = sum(lens)
    out = [torch.full((total + 3, Hkv, 128), 7.0, device=DEV) for _ in range(2)]
    bs.attn_skip_kv_gather(kv, cu_of(lens), None if starts is None else i32(starts), table,
                           total + 3, torch.float32, out=out)
    bs.attn_skip_last_device_error()
    cu = np.concatenate([[0], np.cumsum(lens)])
    for which, got in zip("kv", out):
        got = got.double().cpu().numpy()
        assert (got[total:] == 7.0).all()  # rows behind the last sequence
        for s, e in enumerate(ends):
            want = pool_rows(kv, table, s, max(1, e), which)[e - lens[s]:e]
            np.testing.assert_array_equal(got[cu[s]:cu[s + 1]], want)


def test_gather_reports_bad_rows_and_reads_them_as_zeros():
    kv, table = cache_of("e4m3", [40], 16, 2, 8)
    t = torch.tensor([[0, 0, 0], [99, -5, 0]], dtype=torch.int32, device=DEV)
    t[0] = table[0]
    k, v = bs.attn_skip_kv_gather(kv, i32([0, 3, 20]), i32([-1, 0]), t, 20, torch.float32)
    with pytest.raises(bs.AttnSkipError) as e:
        bs.attn_skip_last_device_error()
    assert e.value.status == bs.ATTN_EINVAL
    assert (k[0] == 0).all() and (v[0] == 0).all() and (k[3:] == 0).all()
    want = pool_rows(kv, table, 0, 2, "k")
    np.testing.assert_array_equal(k[1:3].double().cpu().numpy(), want)
    with pytest.raises(bs.AttnSkipError):  # past the table's last position
        bs.attn_skip_kv_gather(kv, i32([0, 9]), i32([40]), t[:1], 9)
        bs.attn_skip_last_device_error()


# ------------------------------------------------------------------ attend --
def attend(kv, table, chunks, lens, Hq, lams, causal=True, n_splits=1, seed=0, tail=0, q=None,
           scale=0.0, **kw):
    g = np.random.default_rng(seed + 1000)
    total = sum(chunks) + tail
    if q is None:
        q = torch.from_numpy(g.standard_normal((total, Hq, 128))).to(DEV, torch.bfloat16)
    out = bs.attn_skip_chunk_paged(kv, q, cu_of(chunks), max(1, max(chunks)), i32(lens),
                                   max(1, max(lens)), table,
                                   torch.tensor(lams, dtype=torch.float32, device=DEV), causal,
                                   scale, n_splits, with_bits=True, **kw)
    bs.attn_skip_last_device_error()
    return q, out


def check(kv, table, chunks, lens, Hq, lams, q, out, causal=True, n_splits=1, seqs=None,
          scale=128 ** -0.5):
    """Bits equal outside the margin band; outputs, under the GPU's decisions,
    within what the roundings of the computation allow:

    * P is rounded to bf16 (half a step, 2^-8 relative) while the row sum is
      not: at most 2^-8 A in an output element, A = sum p |v|;
    * the output is rounded to bf16: 2^-8 |o|;
    * scores: 128 fp32 products and additions, at most 2^-17 of sum |q k| scale
      (dots) with truncating additions; a score error d moves an output by at
      most 2 d A and the LSE by d;
    * exponentials and the merge: a few fp32 steps of the argument, 2^-18 A."""
    o, lse, bits = out
    G, Hkv = Hq // kv.Hkv, kv.Hkv
    tt = 128 // G
    nb = -(-max(1, max(lens)) // 128)
    bps = -(-nb // n_splits)
    bits = bs.unpack_bits(bits, bps).numpy()  # [n_seq, Hkv, n_t, splits, bps]
    cu = np.concatenate([[0], np.cumsum(chunks)])
    skipped = 0
    for s in (range(len(chunks)) if seqs is None else seqs):
        n, L = chunks[s], lens[s]
        nt = -(-n // tt)
        assert not bits[s, :, nt:].any()
        if n == 0:
            continue
        k, v = (pool_rows(kv, table, s, L, w) if L else np.zeros((0, Hkv, 128)) for w in "kv")
        qs = q[cu[s]:cu[s + 1]].double().cpu().numpy().reshape(n, Hkv, G, 128)
        lam = float(torch.tensor(lams[s], dtype=torch.float32))
        gb = bits[s][:, :nt]
        r = plain.attend(qs, k, v, n, L, G, lam, causal, scale, bps,
                         force=gb)
        if lam > 0:
            # The rule's decisions: the margins do not depend on the skips.
            rule = np.where(np.isnan(r["margin"]), False, r["margin"] < np.log(lam))
            n_bad, _ = compare_bits(gb, rule, r["margin"], lam, label=f"paged lambda={lam:.3g}")
            assert n_bad == 0, f"sequence {s}: {n_bad} bits differ outside the band"
            skipped += int(gb.sum())
        else:
            assert not gb[np.isfinite(r["margin"])].any()
        got = o[cu[s]:cu[s + 1]].double().cpu().numpy().reshape(n, Hkv, G, 128)
        gl = lse[cu[s]:cu[s + 1]].double().cpu().numpy().reshape(n, Hkv, G)
        empty = np.isneginf(r["lse"])
        assert (np.isneginf(gl) == empty).all() and (got[empty] == 0).all()
        d = 2.0 ** -17 * r["dots"]
        tol = (2.0 ** -8 * (r["absv"] * 1.01 + np.abs(r["o"]) * 1.01)
               + (2 * d[..., None] + 2.0 ** -18) * r["absv"])
        err = np.abs(got - r["o"])
        assert (err <= tol).all(), f"sequence {s}: O off by {(err / np.maximum(tol, 1e-300)).max():.3g} of the bound"
        le = np.abs(np.where(empty, 0, gl - np.where(empty, 0, r["lse"])))
        lt = d + 2.0 ** -20 * (8 + np.abs(np.where(empty, 0, r["lse"])))
        assert (le <= lt).all(), f"sequence {s}: LSE off by {(le / lt).max():.3g} of the bound"
    return skipped


CASES = [
    # (chunks, lens, page, Hkv, G, splits)
    ((1,), (1,), 16, 1, 1, 1),
    ((1,), (129,), 16, 2, 4, 2),
    ((1, 1, 1), (127, 128, 1000), 32, 2, 8, 3),
    ((5, 0, 1, 2), (300, 40, 513, 2), 64, 2, 4, 1),
    ((128,), (128,), 128, 1, 1, 1),
    ((33, 97, 200), (33, 640, 300), 64, 2, 4, 1),
    ((300,), (1300,), 256, 1, 3, 1),     # 42 tokens of 3 heads: 126 rows of 128
    ((40, 7), (700, 260), 16, 1, 5, 4),
    ((9,), (900,), 16, 1, 128, 2),       # one token a tile
    ((26,), (257,), 32, 2, 16, 1),
    ((2, 3), (0, 2), 16, 1, 2, 1),       # an empty cache; a chunk longer than its cache
    ((4, 6), (0, 3), 16, 1, 2, 2),
    ((130,), (1,), 16, 1, 1, 1),
    ((3, 7), (500, 900), 384, 2, 4, 3),  # a page size that is no power of two, not four whole parts
    ((1, 2), (400, 260), 16, 1, 16, 2),  # 32 rows
    ((20, 9), (1030, 300), 64, 2, 4, 2),  # 80 rows of one tile
    ((60, 33), (700, 256), 32, 1, 4, 1),  # two tiles
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal", [True, False])
def test_chunk_dense(fmt, case, causal):
    chunks, lens, ps, Hkv, G, n = CASES[case]
    kv, table = cache_of(fmt, lens, ps, Hkv, case)
    lams = [0.0] * len(lens)
    q, out = attend(kv, table, chunks, lens, Hkv * G, lams, causal, n, case)
    check(kv, table, chunks, lens, Hkv * G, lams, q, out, causal, n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("chunks,lens,G,n_splits,lams,some", [
    ((1, 1, 1), (3000, 1111, 640), 4, 1, (0.02, 1e-3, 0.3), True),
    ((200, 64, 3), (1500, 2100, 4000), 8, 1, (0.02, 1e-3, 0.3), True),
    ((50, 1), (5000, 4000), 4, 5, (0.02, 1e-3), False),  # salient keys in every split: none
    ((1, 1), (5000, 4000), 4, 4, (0.5, 0.4), True),
    ((3, 2, 1), (3000, 1111, 640), 8, 1, (0.02, 1e-2, 0.3), True),  # 24 rows
    ((3, 2), (5000, 4000), 8, 3, (0.6, 0.5), False),
    ((20, 4), (3000, 2222), 4, 1, (0.02, 0.1), True),               # 80 rows of one tile
])
def test_chunk_skips_by_the_threshold(fmt, chunks, lens, G, n_splits, lams, some):
    Hkv = 2
    kv, table = cache_of(fmt, lens, 32, Hkv, 40 + G, sink=1.0)
    g = np.random.default_rng(9)
    q = torch.from_numpy(g.standard_normal((sum(chunks), Hkv * G, 128)) + 0.7).to(DEV, torch.bfloat16)
    q, out = attend(kv, table, chunks, lens, Hkv * G, lams, True, n_splits, q=q)
    skipped = check(kv, table, chunks, lens, Hkv * G, lams, q, out, True, n_splits)
    assert skipped > 0 or not some


def test_chunk_rows_behind_the_last_sequence_and_strided_queries():
    chunks, lens, Hkv, G = (3, 18), (500, 90), 2, 4
    Hq, total = Hkv * G, 21 + 5
    kv, table = cache_of("e4m3", lens, 64, Hkv, 50)
    fused = torch.randn(total, Hq + 2 * Hkv, 128, device=DEV).to(torch.bfloat16)
    q = fused[:, :Hq]
    for n in (1, 4):
        bits = torch.full(bs.chunk_bitmap_shape(2, Hq, Hkv, 18, 500, n), -1, dtype=torch.int32,
                          device=DEV)
        o = torch.full((total, Hq, 128), 3.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((total, Hq), 5.0, device=DEV)
        q, out = attend(kv, table, chunks, lens, Hq, [0.0, 0.0], q=q, n_splits=n, tail=5,
                        out=(o, lse, bits))
        assert (o[21:] == 3.0).all() and (lse[21:] == 5.0).all()
        check(kv, table, chunks, lens, Hq, [0.0, 0.0], q, out, n_splits=n)


@pytest.mark.parametrize("n_splits", [1, 2])
def test_chunk_many_sequences(n_splits):
    g = np.random.default_rng(12)
    lens = [int(x) for x in g.integers(1, 400, 77)]
    chunks = [int(min(L, c)) for L, c in zip(lens, g.choice([0, 1, 1, 2, 40], 77))]
    kv, table = cache_of("bf16", lens, 16, 1, 13)
    q, out = attend(kv, table, chunks, lens, 4, [0.0] * 77, n_splits=n_splits)
    check(kv, table, chunks, lens, 4, [0.0] * 77, q, out, n_splits=n_splits)


def batch(n, longest, seed, kinds=(1, 1, 1, 2)):
    """n sequences of mixed lengths, some of them empty, one of them the longest."""
    g = np.random.default_rng(seed)
    lens = [int(x) for x in g.integers(1, longest, n)]
    chunks = [int(c) for c in g.choice(kinds, n)]
    lens[n // 2], lens[n // 3], lens[n - 1], chunks[n // 4] = longest, 0, 1, 0
    return chunks, lens


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("n,longest,Hkv,G,n_splits", [
    (24, 2500, 4, 4, 7),    # tiles cut where the CTAs' runs end
    (3, 9000, 8, 1, 20),    # few long tiles: a run per block
    (40, 130, 4, 2, 2),     # two blocks at most
    (100, 300, 4, 4, 1),    # whole tiles, several a CTA
    (33, 1500, 2, 3, 64),   # more slots than blocks
    (128, 700, 1, 4, 3),
    (129, 700, 1, 4, 3),    # more sequences than are shared out
])
def test_decode_of_more_pieces_than_ctas(fmt, n, longest, Hkv, G, n_splits):
    assert n * Hkv * n_splits > 304
    chunks, lens = batch(n, longest, n + G)
    kv, table = cache_of(fmt, lens, 16, Hkv, n)
    q, out = attend(kv, table, chunks, lens, Hkv * G, [0.0] * n, n_splits=n_splits, seed=n)
    check(kv, table, chunks, lens, Hkv * G, [0.0] * n, q, out, n_splits=n_splits)
    again = attend(kv, table, chunks, lens, Hkv * G, [0.0] * n, n_splits=n_splits, q=q)[1]
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("n,longest,n_splits", [(24, 2500, 7), (100, 400, 2), (160, 200, 1)])
def test_decode_of_more_pieces_than_ctas_skips(fmt, n, longest, n_splits):
    """Thresholds on some sequences: the splits' bounds hold for every tile."""
    Hkv, G = 2, 4
    chunks, lens = batch(n, longest, n)
    lams = [(0.0, 0.3, 0.6)[s % 3] for s in range(n)]
    kv, table = cache_of(fmt, lens, 32, Hkv, n, sink=1.0)
    g = np.random.default_rng(n)
    q = torch.from_numpy(g.standard_normal((sum(chunks), Hkv * G, 128)) + 0.7).to(DEV, torch.bfloat16)
    q, out = attend(kv, table, chunks, lens, Hkv * G, lams, True, n_splits, q=q)
    skipped = check(kv, table, chunks, lens, Hkv * G, lams, q, out, True, n_splits)
    assert skipped > 0


@pytest.mark.parametrize("n_splits", [1, 4])
def test_decode_of_more_pieces_than_ctas_with_bad_device_arguments(n_splits):
    n, Hkv, Hq = 110, 3, 6
    lens = [200 + s for s in range(n)]
    kv, table = cache_of("e4m3", lens, 16, Hkv, 14)
    q = torch.randn(n + 4, Hq, 128, device=DEV).to(torch.bfloat16)
    cu, kl, lam = i32(range(n + 1)), i32(lens), torch.zeros(n, device=DEV)
    want, wl, _ = bs.attn_skip_chunk_paged(kv, q, cu, 1, kl, max(lens), table, lam, n_splits=n_splits)
    bs.attn_skip_last_device_error()
    bad_cu, bad_kl, bad_t, bad_lam = cu.clone(), kl.clone(), table.clone(), lam.clone()
    bad_cu[41:] += 1                       # sequence 40: two tokens, one allowed
    bad_kl[7], bad_kl[50] = max(lens) + 1, -1
    bad_t[3, 2], bad_t[3, 5] = -4, 10 ** 6
    bad_lam[9] = float("nan")
    o, lse = torch.full_like(want, 2.0), torch.full_like(wl, 2.0)
    bs.attn_skip_chunk_paged(kv, q, bad_cu, 1, bad_kl, max(lens), bad_t, bad_lam, n_splits=n_splits,
                             out=(o, lse, None))
    with pytest.raises(bs.AttnSkipError) as e:
        bs.attn_skip_last_device_error()
    assert e.value.status == bs.ATTN_EINVAL
    for s in (7, 50):
        r = s + (s > 40)
        assert (o[r] == 0).all() and torch.isneginf(lse[r]).all()
    for r in (40, 41, n + 1, n + 2, n + 3):  # the sequence left out; rows behind the last one
        assert (o[r] == 2).all() and (lse[r] == 2).all()
    for s in (0, 1, 2, 4, 9, 39):
        assert torch.allclose(o[s].float(), want[s].float(), atol=0.02)


PROMPTS = [
    # (sequences, longest chunk, tokens before it, Hkv, G, splits): more tiles than SMs
    (40, 200, 300, 2, 4, 1),
    (30, 150, 500, 2, 7, 3),    # 126 rows a tile, splits without a block
    (10, 40, 90, 1, 128, 1),    # a tile a token
    (70, 60, 0, 2, 16, 2),
    (100, 33, 100, 4, 3, 1),    # one tile a sequence, partly filled quarters
]


def prompts(case):
    n, longest, before, Hkv, G, n_splits = PROMPTS[case]
    g = np.random.default_rng(case)
    chunks = [int(c) for c in g.integers(0, longest + 1, n)]
    chunks[1], chunks[2] = longest, 0
    lens = [int(c + g.integers(0, before + 1)) for c in chunks]
    lens[3], lens[4] = 0, max(0, chunks[4] - 2)  # an empty cache; a chunk longer than its cache
    tt = 128 // G
    assert sum(-(-c // tt) for c in chunks) * Hkv * n_splits > 152
    return chunks, lens, Hkv, G, n_splits


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_of_many_tiles(fmt, case, causal):
    chunks, lens, Hkv, G, n = prompts(case)
    kv, table = cache_of(fmt, lens, 32, Hkv, case)
    lams = [0.0] * len(lens)
    q, out = attend(kv, table, chunks, lens, Hkv * G, lams, causal, n, case)
    check(kv, table, chunks, lens, Hkv * G, lams, q, out, causal, n)
    again = attend(kv, table, chunks, lens, Hkv * G, lams, causal, n, q=q)[1]
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompts_of_many_tiles_skip(case):
    chunks, lens, Hkv, G, n = prompts(case)
    kv, table = cache_of("bf16", lens, 64, Hkv, case, sink=1.0)
    lams = [(0.0, 0.3, 0.6)[s % 3] for s in range(len(lens))]
    g = np.random.default_rng(case)
    q = torch.from_numpy(g.standard_normal((sum(chunks), Hkv * G, 128)) + 0.7).to(DEV, torch.bfloat16)
    q, out = attend(kv, table, chunks, lens, Hkv * G, lams, True, n, q=q)
    check(kv, table, chunks, lens, Hkv * G, lams, q, out, True, n)


def test_prompts_of_many_tiles_with_bad_device_arguments():
    n, Hkv, Hq, C = 60, 2, 8, 70
    lens = [C + s for s in range(n)]
    kv, table = cache_of("bf16", lens, 16, Hkv, 15)
    q = torch.randn(n * C + 5, Hq, 128, device=DEV).to(torch.bfloat16)
    cu, kl, lam = i32(range(0, n * C + 1, C)), i32(lens), torch.zeros(n, device=DEV)
    args = dict(max_chunk=C, max_kv=max(lens), n_splits=1)
    want, wl, _ = bs.attn_skip_chunk_paged(kv, q, cu, kv_len=kl, page_table=table, lambdas=lam, **args)
    bs.attn_skip_last_device_error()
    bad_cu, bad_kl, bad_t, bad_lam = cu.clone(), kl.clone(), table.clone(), lam.clone()
    bad_cu[31:] += 1                     # sequence 30: 71 tokens, 70 allowed
    bad_kl[7], bad_kl[50] = max(lens) + 1, -1
    bad_t[3, 2], bad_t[3, 4] = -4, 10 ** 6
    bad_lam[9] = float("nan")
    o, lse = torch.full_like(want, 2.0), torch.full_like(wl, 2.0)
    bs.attn_skip_chunk_paged(kv, q, bad_cu, kv_len=bad_kl, page_table=bad_t, lambdas=bad_lam,
                             out=(o, lse, None), **args)
    with pytest.raises(bs.AttnSkipError) as e:
        bs.attn_skip_last_device_error()
    assert e.value.status == bs.ATTN_EINVAL
    for s in (7, 50):
        r = slice(s * C + (s > 30), (s + 1) * C + (s > 30))
        assert (o[r] == 0).all() and torch.isneginf(lse[r]).all()
    assert (o[30 * C:31 * C + 1] == 2).all() and (lse[30 * C:31 * C + 1] == 2).all()
    assert (o[n * C + 1:] == 2).all() and (lse[n * C + 1:] == 2).all()
    for s in (0, 1, 2, 4, 9, 29):
        assert torch.equal(o[s * C:(s + 1) * C], want[s * C:(s + 1) * C])


@pytest.mark.parametrize("ps", [128, 256, 384])
@pytest.mark.parametrize("fmt,n,C,G,n_splits", [
    ("e4m3", 20, 2, 4, 9), ("nvfp4", 20, 1, 8, 9), ("bf16", 20, 90, 4, 1), ("bf16", 20, 90, 4, 3),
    ("e4m3", 20, 100, 4, 2), ("bf16", 60, 3, 4, 2),
])
def test_large_batches_share_pages_of_many_rows(fmt, ps, n, C, G, n_splits):
    """Grids of more pieces or tiles than the chip takes at once, over pages of one
    to three blocks; every sequence stands twice in the batch, on the same pages."""
    Hkv, g = 2, np.random.default_rng(n + ps)
    lens = [int(x) for x in g.integers(max(C, 700), 1400, n // 2)]
    chunks = [int(x) for x in g.integers(1, C + 1, n)]
    kv, table = cache_of(fmt, lens, ps, Hkv, n)
    lens, table = lens + lens, torch.cat([table, table]).contiguous()
    q, out = attend(kv, table, chunks, lens, Hkv * G, [0.0] * n, n_splits=n_splits, seed=ps)
    check(kv, table, chunks, lens, Hkv * G, [0.0] * n, q, out, n_splits=n_splits)


@pytest.mark.parametrize("fmt,n,C", [("bf16", 40, 100), ("e4m3", 64, 1), ("bf16", 3, 60)])
def test_a_workspace_serves_calls_of_any_kind(fmt, n, C):
    """What one call leaves in the partials means nothing to the next: dense calls and
    calls with thresholds, sound ones and ones with a bad sequence, in turn."""
    Hkv, Hq, L, ns = 2, 8, 900, 3
    kv, table = cache_of(fmt, [L] * n, 32, Hkv, n, sink=1.0)
    cu, kl = i32(range(0, n * C + 1, C)), i32([L] * n)
    q = (torch.randn(n * C, Hq, 128, device=DEV) + 0.7).to(torch.bfloat16)
    dense = torch.zeros(n, device=DEV)
    some = torch.where(torch.arange(n, device=DEV) % 2 == 0, 0.5, 0.0)
    short = kl.clone()
    short[0] = 0
    calls = [(cu, kl, dense), (cu, kl, some), (cu, short, dense), (cu, short, some), (cu, kl, dense)]
    work = (torch.full((n * C, Hq, ns, 128), float("nan"), device=DEV),
            torch.full((n * C, Hq, ns), float("nan"), device=DEV))
    for c, k, lam in calls:
        want = bs.attn_skip_chunk_paged(kv, q, c, C, k, L, table, lam, n_splits=ns)
        got = bs.attn_skip_chunk_paged(kv, q, c, C, k, L, table, lam, n_splits=ns, workspace=work)
        bs.attn_skip_last_device_error()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.isfinite(got[0].float()).all()


@pytest.mark.parametrize("fmt,n,C,L", [("bf16", 40, 100, 400), ("nvfp4", 64, 1, 1500)])
def test_large_batches_on_two_streams_and_in_a_graph(fmt, n, C, L):
    """Grids whose CTAs take over one another's work, or share it out, next to
    each other."""
    kv, table = cache_of(fmt, [L] * n, 16, 2, 3)
    cu, kl, lam = i32(range(0, n * C + 1, C)), i32([L] * n), torch.zeros(n, device=DEV)
    qs = [torch.randn(n * C, 8, 128, device=DEV).to(torch.bfloat16) for _ in range(2)]

    def call(q, **kw):
        return bs.attn_skip_chunk_paged(kv, q, cu, C, kl, L, table, lam, n_splits=3, **kw)[:2]

    want = [call(q) for q in qs]
    bs.attn_skip_last_device_error()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[call(q, stream=st) for _ in range(3)] for q, st in zip(qs, streams) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [call(q) for q in qs]
    for _ in range(2):
        graph.replay()
    bs.attn_skip_last_device_error()
    for i, calls in enumerate(got):
        for o, lse in calls:
            assert torch.equal(o, want[i // 2][0]) and torch.equal(lse, want[i // 2][1])
    for (o, lse), (wo, wl) in zip(captured, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("fmt", FORMATS)
def test_chunk_scale_and_large_values(fmt):
    """An explicit score scale, and rows whose scale byte needs a second bf16
    factor in the widening (values above 57344)."""
    lens = (200,)
    kv, table = cache_of(fmt, lens, 64, 1, 60, scale=2e5)
    q = (torch.randn(3, 2, 128, device=DEV) * 1e-5).to(torch.bfloat16)
    sc = 0.05
    q, out = attend(kv, table, (3,), lens, 2, [0.0], q=q, scale=sc)
    check(kv, table, (3,), lens, 2, [0.0], q, out, scale=sc)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "bf16"])
@pytest.mark.parametrize("Hq", [2, 8, 40])  # 4, 16 and 80 rows
def test_chunk_nan_row_reaches_the_rows_that_see_it(fmt, Hq):
    kv, table = cache_of(fmt, (300, 300), 16, 1, 61)
    bad = torch.full((1, 1, 128), float("nan"), device=DEV)
    good = torch.ones(1, 1, 128, device=DEV)
    # Position 299 of sequence 0 gets a NaN key.
    bs.attn_skip_kv_append(kv, bad, good, i32([0, 1, 1]), i32([300, 300]), table)
    q, (o, lse, _) = attend(kv, table, (2, 2), (300, 300), Hq, [0.0, 0.0])
    assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[2:]).all()  # it is masked, or another's


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("chunks,Hq", [((2, 1), 4), ((4, 3), 4), ((40, 9), 4), ((200, 90), 4)])
def test_chunk_rows_of_very_different_scales(fmt, chunks, Hq):
    """Small rows next to rows of zeros (whose scale byte is 127) and rows 2^12
    apart: one exponent a block has to serve them all."""
    lens, g = (300, 260), np.random.default_rng(63)
    table, n_pages = tables(lens, 16, g)
    kv = filled_cache(fmt, n_pages, 16, 1)
    x = [g.standard_normal((560, 1, 128)) * 2.0 ** -17 for _ in range(2)]
    for y in x:
        y[g.random(560) < 0.1] = 0.0
        y[g.random(560) < 0.3] *= 2.0 ** -12
    k, v = (torch.from_numpy(y).to(DEV, torch.float32) for y in x)
    bs.attn_skip_kv_append(kv, k, v, cu_of(lens), i32(lens), table)
    q = (torch.randn(sum(chunks), Hq, 128, device=DEV) * 2.0 ** 17).to(torch.bfloat16)
    q, out = attend(kv, table, chunks, lens, Hq, [0.0, 0.0], q=q)
    check(kv, table, chunks, lens, Hq, [0.0, 0.0], q, out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 7, 20])  # 4, 28 and 80 rows
def test_chunk_distant_key_behind_zeros(fmt, n):
    """Where the key with all the weight has a value of zero, an output is what a
    key 13.6 nats below it brings: it is as exact as any other."""
    Hkv, G = 1, 4
    kv = filled_cache(fmt, 2, 16, Hkv)
    table = i32([1]).view(1, 1)
    k = torch.ones(3, Hkv, 128, device=DEV, dtype=torch.bfloat16)
    k[0], k[2] = -1, 0.5
    v = torch.randn(3, Hkv, 128, device=DEV).to(torch.bfloat16)
    v[1, :, ::2], v[2] = 0, 0
    bs.attn_skip_kv_append(kv, k, v, cu_of([3]), i32([3]), table)
    q = torch.full((n, Hkv * G, 128), 0.6, device=DEV, dtype=torch.bfloat16)
    q, out = attend(kv, table, (n,), (3,), Hkv * G, [0.0], False, q=q)
    check(kv, table, (n,), (3,), Hkv * G, [0.0], q, out, False)


def test_chunk_reports_bad_device_arguments():
    kv, table = cache_of("e4m3", (300, 200, 100), 16, 1, 62)
    q = torch.randn(9, 4, 128, device=DEV).to(torch.bfloat16)
    lam = torch.zeros(3, device=DEV)
    want, wl, _ = bs.attn_skip_chunk_paged(kv, q, i32([0, 3, 6, 9]), 3, i32([300, 200, 100]), 300,
                                           table, lam, n_splits=1)
    bs.attn_skip_last_device_error()

    def bad(cu=(0, 3, 6, 9), lens=(300, 200, 100), t=table, lam=lam, n_splits=1, max_chunk=3):
        o = torch.full_like(want, 2.0)
        lse = torch.full_like(wl, 2.0)
        bs.attn_skip_chunk_paged(kv, q, i32(cu), max_chunk, i32(lens), 300, t, lam, n_splits=n_splits,
                                 out=(o, lse, None))
        with pytest.raises(bs.AttnSkipError) as e:
            bs.attn_skip_last_device_error()
        assert e.value.status == bs.ATTN_EINVAL
        bs.attn_skip_last_device_error()
        return o, lse

    for n in (1, 3):
        t = table.clone()
        t[0, 5], t[0, 9] = 100000, -7
        o, _ = bad(t=t, n_splits=n)
        assert torch.allclose(o[3:].float(), want[3:].float(), atol=0.02)
        o, lse = bad(lens=(301, 200, 100), n_splits=n)  # beyond max_kv: an empty cache
        assert (o[:3] == 0).all() and torch.isneginf(lse[:3]).all()
        assert torch.allclose(o[3:].float(), want[3:].float(), atol=0.02)
        o, lse = bad(lens=(300, -1, 100), n_splits=n)
        assert (o[3:6] == 0).all()
        o, lse = bad(cu=(0, 3, 7, 9), n_splits=n)  # 4 tokens, max_chunk 3: not written
        assert (o[3:7] == 2).all() and (lse[3:7] == 2).all() and (o[:3] != 2).any()
        o, _ = bad(cu=(0, 3, 6, 10), n_splits=n, max_chunk=4)
        assert (o[6:] == 2).all()
        o, _ = bad(cu=(0, 3, 2, 5), n_splits=n)  # decreasing bounds: that sequence is left out
    for v in (1.0, -0.5, float("nan")):
        o, _ = bad(lam=torch.tensor([0.0, v, 0.0], device=DEV))  # treated as 0
        assert torch.equal(o, want)


def test_offsets_beyond_32_bits():
    """Pools of more than 2^32 bytes: the last pages are written, read and attended."""
    ps, Hkv = 128, 8
    n_pages = (1 << 32) // (Hkv * ps * 256) * 2 + 5  # k and v of 8.6 GB each
    for fmt in ("bf16", "e4m3"):
        n = n_pages if fmt == "bf16" else 2 * n_pages
        kv = bs.PagedKV.empty(fmt, n, ps, Hkv, device=DEV)
        L = 300
        table = torch.tensor([[n - 1, n // 2 + 3, n - 2]], dtype=torch.int32, device=DEV)
        k, v = (torch.randn(L, Hkv, 128, device=DEV).to(torch.bfloat16) for _ in range(2))
        bs.attn_skip_kv_append(kv, k, v, i32([0, L]), i32([L]), table)
        ref = bs.PagedKV.empty(fmt, 3, ps, Hkv, device=DEV)
        rt = torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV)
        bs.attn_skip_kv_append(ref, k, v, i32([0, L]), i32([L]), rt)
        a = bs.attn_skip_kv_gather(kv, i32([0, L]), None, table, L)
        b = bs.attn_skip_kv_gather(ref, i32([0, L]), None, rt, L)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        q = torch.randn(40, 16, 128, device=DEV).to(torch.bfloat16)
        lam = torch.zeros(1, device=DEV)
        x = bs.attn_skip_chunk_paged(kv, q, i32([0, 40]), 40, i32([L]), L, table, lam)
        y = bs.attn_skip_chunk_paged(ref, q, i32([0, 40]), 40, i32([L]), L, rt, lam)
        bs.attn_skip_last_device_error()
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        del kv


@pytest.mark.parametrize("fmt", FORMATS)
def test_keys_and_values_in_one_pool(fmt):
    """Pages that hold keys and values next to each other."""
    Hkv, ps, L = 2, 32, 100
    ref, table = cache_of(fmt, (L,), ps, Hkv, 70)
    both = torch.empty(ref.n_pages, 2, *ref.k.shape[1:], dtype=ref.k.dtype, device=DEV)
    kv = bs.PagedKV(fmt, both[:, 0], both[:, 1], ref.k_scale, ref.v_scale, ref.k_bs, ref.v_bs)
    both[:, 0], both[:, 1] = ref.k, ref.v
    q, a = attend(ref, table, (5,), (L,), 4, [0.0])
    _, b = attend(kv, table, (5,), (L,), 4, [0.0], q=q)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    new = torch.randn(7, Hkv, 128, device=DEV)
    for c in (ref, kv):
        bs.attn_skip_kv_append(c, new, new, i32([0, 7]), i32([L]), table)
    x = bs.attn_skip_kv_gather(ref, i32([0, L]), None, table, L)
    y = bs.attn_skip_kv_gather(kv, i32([0, L]), None, table, L)
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_conversation(fmt):
    """As a serving loop uses them: a prompt in two chunks, then tokens one by
    one, two sequences of different lengths; each step's outputs against the
    plain attention over the rows that the cache holds."""
    Hkv, G, ps = 2, 4, 16
    Hq = Hkv * G
    g = np.random.default_rng(80)
    table, n_pages = tables((400, 300), ps, g)
    kv = filled_cache(fmt, n_pages, ps, Hkv)
    lens = [0, 0]
    for step, chunks in enumerate(((130, 70), (200, 0), (1, 1), (1, 1), (3, 2))):
        lens = [a + b for a, b in zip(lens, chunks)]
        total = sum(chunks)
        qkv = torch.from_numpy(g.standard_normal((total, Hq + 2 * Hkv, 128))).to(DEV, torch.bfloat16)
        bs.attn_skip_kv_append(kv, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cu_of(chunks), i32(lens),
                               table)
        n = 2 if max(chunks) < 4 else 1
        q, out = attend(kv, table, chunks, lens, Hq, [0.0, 0.0], q=qkv[:, :Hq], n_splits=n)
        check(kv, table, chunks, lens, Hq, [0.0, 0.0], q, out, n_splits=n)


def test_whole_prompt_equals_the_prefill():
    """A prompt that is its own chunk, against attn_skip_prefill on the same
    rows: both within P's and the output's roundings of the same value."""
    T, Hkv, G = 1000, 2, 4
    q, k, v = (torch.randn(T, h, 128, device=DEV).to(torch.bfloat16) for h in (Hkv * G, Hkv, Hkv))
    table, n_pages = tables((T,), 64, np.random.default_rng(1))
    kv = filled_cache("bf16", n_pages, 64, Hkv)
    bs.attn_skip_kv_append(kv, k, v, i32([0, T]), i32([T]), table)
    o, lse, _ = bs.attn_skip_chunk_paged(kv, q, i32([0, T]), T, i32([T]), T, table,
                                         torch.zeros(1, device=DEV))
    p, pl, _ = bs.attn_skip_prefill(*(x.transpose(0, 1)[None].contiguous() for x in (q, k, v)), 0.0)
    bs.attn_skip_last_device_error()
    # Each is off by at most 2^-8 (A + |o|) with A = sum p |v| <= max |v|.
    d = (o.transpose(0, 1).double() - p[0].double()).abs()
    assert (d <= 2 * 2.0 ** -8 * 1.01 * (v.abs().max().double() + p[0].double().abs())).all()
    assert (lse.T - pl[0]).abs().max() <= 2.0 ** -14


# ------------------------------------------------- streams, graphs, repeats --
def decode_state(fmt, seed=90):
    kv, table = cache_of(fmt, (700, 333), 16, 2, seed)
    q = torch.randn(2, 8, 128, device=DEV).to(torch.bfloat16)
    return kv, table, q, torch.zeros(2, device=DEV)


@pytest.mark.parametrize("fmt", FORMATS)
def test_repeats_are_identical_and_queue_up(fmt):
    kv, table, q, lam = decode_state(fmt)
    outs = [bs.attn_skip_chunk_paged(kv, q, i32([0, 1, 2]), 1, i32([700, 333]), 700, table, lam,
                                     n_splits=n) for n in (3,) * 12]
    bs.attn_skip_last_device_error()
    for o, lse, _ in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_another_stream():
    kv, table, q, lam = decode_state("e4m3")
    cu, lens = i32([0, 1, 2]), i32([700, 333])
    want = bs.attn_skip_chunk_paged(kv, q, cu, 1, lens, 700, table, lam, n_splits=4)
    rows = bs.attn_skip_kv_gather(kv, i32([0, 20, 40]), None, table, 40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for st in (side, side.cuda_stream):
        got = bs.attn_skip_chunk_paged(kv, q, cu, 1, lens, 700, table, lam, n_splits=4, stream=st)
        back = bs.attn_skip_kv_gather(kv, i32([0, 20, 40]), None, table, 40, stream=st)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])


def test_captured_steps_follow_the_device_lengths():
    """A step captured once and replayed as the sequences grow: lengths and the
    page table are device data.  Two graphs with a workspace of their own."""
    Hkv, Hq, ps = 2, 8, 16
    g = np.random.default_rng(95)
    table, n_pages = tables((200, 200), ps, g)
    kv, ref = filled_cache("nvfp4", n_pages, ps, Hkv), filled_cache("nvfp4", n_pages, ps, Hkv)
    lens, cu = i32([100, 57]), i32([0, 1, 2])
    k0 = torch.randn(157, Hkv, 128, device=DEV).to(torch.bfloat16)
    for c in (kv, ref):
        bs.attn_skip_kv_append(c, k0, k0, i32([0, 100, 157]), lens, table)
    qkv = torch.zeros(2, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device=DEV)
    lam = torch.zeros(2, device=DEV)

    def step(c):
        bs.attn_skip_kv_append(c, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], cu, lens, table)
        return bs.attn_skip_chunk_paged(c, qkv[:, :Hq], cu, 1, lens, 200, table, lam, n_splits=2)
    for c in (ref, kv):  # the first calls load the kernels before the capture
        step(c)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(kv)
        graphs.append((graph, out))
    for i in range(6):
        lens += 1
        qkv.copy_(torch.randn_like(qkv, dtype=torch.float32))
        want = step(ref)
        graph, out = graphs[i % 2]
        graph.replay()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    bs.attn_skip_last_device_error()


def test_binding_refusals():
    kv, table, q, lam = decode_state("bf16")
    cu, lens = i32([0, 1, 2]), i32([700, 333])
    ok = dict(kv=kv, q=q, cu_seqlens=cu, max_chunk=1, kv_len=lens, max_kv=700, page_table=table,
              lambdas=lam)
    for kw in (dict(q=q.float()), dict(q=q[:, :7]), dict(q=q[:, ::2]), dict(cu_seqlens=cu.long()),
               dict(kv_len=lens[:1]), dict(page_table=table.long()), dict(page_table=table[:1]),
               dict(lambdas=lam.double()), dict(lambdas=lam.cpu()), dict(n_splits=-1),
               dict(n_splits=2, workspace=(lam, lam)), dict(out=(q.float(), lam, None)),
               dict(max_kv=10 ** 6)):
        with pytest.raises((ValueError, TypeError, bs.AttnSkipError)):
            bs.attn_skip_chunk_paged(**{**ok, **kw})
    k = torch.randn(2, 2, 128, device=DEV)
    for a, b in ((k, k[:1]), (k.half(), k.half()), (k[:, :1], k[:, :1]), (k, k.bfloat16()),
                 (k.cpu(), k.cpu())):
        with pytest.raises((ValueError, TypeError)):
            bs.attn_skip_kv_append(kv, a, b, cu, lens, table)
    with pytest.raises(TypeError):
        bs.attn_skip_kv_gather(kv, cu, None, table, 2, torch.float16)
    with pytest.raises(ValueError):
        bs.attn_skip_kv_gather(kv, cu, None, table, 2, out=(k, k))
    bs.attn_skip_last_device_error()
